"""How the work of gathering attention weights is cut into shares, on the CPU.

Every CTA finds its own share from the requests' lengths, in closed form; a
step that two CTAs take, or none, or a part that is added by a CTA that does not
hold it, would only show on a GPU.  A C++ harness (weights_share_dump.cpp) runs
the kernels' share arithmetic, and this test compares what the CTAs take with
the tokens that see each key by definition, counted token by token.
"""
import json
import os
import random
import subprocess

import pytest

import __graft_entry__

__graft_entry__.build()
from gated_rank_subspace_gb300 import _build  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))


def cases():
    rng = random.Random(5)
    out = [(kt, 3, 16, 1, 1, 4, 9, [], []) for kt in (64, 128, 256)]
    for i in range(260):
        kt = rng.choice([64, 128, 256])
        tpt = rng.choice([t for t in (1, 2, 4, 8, 16, 32, 64, 128) if t <= kt])
        n_req = rng.choice([1, 1, 2, 3, 9, 40, 500])
        most_q, most_k = rng.choice([(1, 900), (3, 60), (40, 700), (700, 2000), (300, 100)])
        if n_req >= 40:
            most_q, most_k = min(most_q, 5), min(most_k, 300)
        lens = [(rng.randint(0, most_q), rng.randint(0, most_k)) for _ in range(n_req)]
        if i % 4 == 0:
            q = rng.randint(1, 1500)
            lens = [(q, q + rng.choice([0, 0, 1, 500]))]
        held = [rng.choice([0, k, k + 3, rng.randint(0, k), max(0, k - q)]) for q, k in lens]
        out.append((kt, rng.choice([1, 2, 5, 9, 16, 304 if n_req < 40 else 30]), tpt, rng.choice([1, 2, 3, 5]), int(rng.random() < 0.8), 4, 200, lens, held))
    # requests that add nothing before, between and behind those that do
    out.append((64, 7, 4, 2, 1, 4, 200, [(0, 0), (0, 50), (3, 200), (0, 0), (0, 0), (5, 5), (0, 70), (2, 0), (0, 9)], [0, 50, 197, 0, 0, 0, 10, 0, 9]))
    return out


def steps_of(kt, tpt, causal, q, k, held, t):
    """First row tile with a token that sees a key of tile t, and the number from there on."""
    sees = [i for i in range(q) if not causal or k - q + i >= t * kt]  # token i sees the keys up to its own place
    return (sees[0] // tpt, (q - 1) // tpt + 1 - sees[0] // tpt) if sees else (0, 1)


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("share") / "dump")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    subprocess.run(["g++", "-O1", "-w", "-std=c++17", "-I", cuda, "-I", _build.CSRC, "-I", _build.INCLUDE, os.path.join(HERE, "weights_share_dump.cpp"), "-o", exe], check=True)
    lines = []
    for kt, grid, tpt, hkv, causal, shift, width, lens, held in cases():
        start = [0]
        for q, _ in lens:
            start.append(start[-1] + q)
        lines.append(" ".join(map(str, [kt, grid, tpt, hkv, causal, shift, width, start[-1], len(lens), *start, *(k for _, k in lens), *held])))
    got = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, check=True, timeout=600).stdout.splitlines()
    assert len(got) == len(lines)
    return [json.loads(g) for g in got]


def test_every_step_is_taken_once(answers):
    for (kt, grid, tpt, hkv, causal, _, _, lens, held), got in zip(cases(), answers):
        assert got["alike"] == 1 and len(got["ctas"]) == grid
        want = []
        for r, ((q, k), h0) in enumerate(zip(lens, held)):
            first = 0 if q > 0 else min(h0, k) // kt if h0 < k else -(-k // kt)
            for h in range(hkv):
                want += [(r, h, t, *steps_of(kt, tpt, causal, q, k, h0, t)) for t in range(first, -(-k // kt))]
        taken, holders = {}, {}
        for c, segs in enumerate(got["ctas"]):
            for r, h, t, u0, n, a, b, b0, b1 in segs:
                assert 0 <= a < b <= n
                taken.setdefault((r, h, t, u0, n), []).append((a, b, c, b0, b1))
        assert list(taken) == want  # in the order of the line, each unit once
        for key, parts in taken.items():
            assert [p[0] for p in parts] == [0] + [p[1] for p in parts[:-1]] and parts[-1][1] == key[4]
            if len(parts) > 1:
                assert {(p[3], p[4]) for p in parts} == {(parts[0][2], parts[-1][2])}
                assert [p[2] for p in parts] == list(range(parts[0][2], parts[-1][2] + 1))
                holders.setdefault(parts[0][2], []).append(key)
        assert all(len(v) == 1 for v in holders.values())  # a CTA begins one unit at most that another one ends: a counter each
        sizes = [sum(b - a for _, _, _, _, _, a, b, _, _ in segs) for segs in got["ctas"]]
        some = [s for s in sizes if s]
        assert not some or max(some) - min(some) <= 1
