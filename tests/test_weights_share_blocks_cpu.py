"""The shares of the gathered attention weights as the kernel of many rows finds
them: 128 keys a unit, blocks of 384 threads."""
import os

import test_weights_share_cpu as share

CASES = [c for c in share.cases() if c[0] == 128]


def test_blocks_of_the_kernel_of_many_rows(tmp_path, monkeypatch):
    with open(os.path.join(share.HERE, "weights_share_dump.cpp")) as f:
        source = f.read()
    assert source.count("run<128, 448>") == 1
    (tmp_path / "weights_share_dump.cpp").write_text(source.replace("run<128, 448>", "run<128, 384>"))
    monkeypatch.setattr(share, "HERE", str(tmp_path))
    monkeypatch.setattr(share, "cases", lambda: CASES)

    class Factory:
        @staticmethod
        def mktemp(name):
            (tmp_path / name).mkdir()
            return tmp_path / name
    share.test_every_step_is_taken_once(share.answers.__wrapped__(Factory))
