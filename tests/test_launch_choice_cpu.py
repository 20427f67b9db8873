"""Which kernel a serving call launches, and with what, without a GPU.

A small C++ harness (fake_runtime.cpp) runs the built library against a fake of
the runtime calls on a launch's path.  A kernel that is launched for a shape
it has no unit for would only show on a GPU, as a fault.
"""
import json
import os
import shutil
import subprocess

import pytest

import __graft_entry__

__graft_entry__.build()
from gated_rank_subspace_gb300 import _build  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not available")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    exe = str(tmp_path_factory.mktemp("fake") / "fake_runtime")
    subprocess.run([gxx, "-std=c++17", "-O1", "-rdynamic", "-I", _build.INCLUDE, "-I", os.path.join(cuda, "include"),
                    os.path.join(HERE, "fake_runtime.cpp"), _build.LIB, "-Wl,-rpath," + os.path.dirname(_build.LIB),
                    "-Wl,-rpath," + os.path.join(cuda, "lib64"), "-L" + os.path.join(cuda, "lib64"), "-lcudart", "-ldl",
                    "-o", exe], check=True)

    def go(*commands):
        r = subprocess.run([exe], input="\n".join(commands) + "\n", capture_output=True, text=True, check=True)
        return [json.loads(x) for x in r.stdout.splitlines()]

    return go


def attention(dt, group, N, max_q, hkv=2, dim=64, n_req=1, width=8, page=16, window=0):
    return f"attention {dt} {group} {hkv} {dim} {N} {max_q} {n_req} {width} {page} {window}"


HINTS = [0, 1, 2, 5, 300, 2**31, 2**62, 2**63 - 1]


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("group", [1, 2, 8, 9, 16, 17, 32, 64, 65, 128])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_attention_kernel_holds_a_token_of_the_group(run, dt, group, dim):
    # a unit of the few-row kernels is 8 / group (float32: 16 / group) tokens: at least one, whatever the caller's hint says
    N = 5
    for hint, r in zip(HINTS, run(*[attention(dt, group, N, h, dim=dim) for h in HINTS])):
        assert r["status"] == 0
        (launch,) = r["launches"]
        name = launch["kernel"]
        if "attn_rows_kernel" in name:
            assert group <= 8, (hint, name)
        elif "attn_f32_kernelILi16" in name:
            assert group <= 16, (hint, name)
        elif "attn_f32_kernelILi64" in name:
            assert group <= 64, (hint, name)
        elif "attn_tiles_kernel" in name:
            assert group <= 128
        else:
            assert "attn_plain_kernel" in name and dt == F32


@pytest.mark.parametrize("group", [1, 4, 8, 9, 16, 64, 128])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_attention_hint_beyond_the_tokens_is_their_number(run, dt, group):
    # no hint below one token or above all of them can mean anything else
    a = run(*[attention(dt, group, 300, h) for h in (0, 1, 300, 301, 2**31, 2**62, 2**63 - 1)])
    names = [r["launches"][0]["kernel"] for r in a]
    assert names[0] == names[1] and len(set(names[2:])) == 1


CALLS = {"rows": attention(BF16, 1, 4, 1), "rows, 256 columns": attention(BF16, 1, 4, 1, dim=256),
         "tiles": attention(BF16, 1, 600, 600), "tiles, 256 columns": attention(BF16, 4, 600, 600, dim=256),
         "float32, few rows": attention(F32, 1, 4, 1, dim=256), "float32": attention(F32, 1, 6000, 6000, dim=128, width=512),
         "plan": "plan 40 40000", "norm, registers": "norm 4000 5120", "norm, shared memory": "norm 4000 5128"}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_every_device_is_set_up(run, call):
    # what a kernel may have of shared memory, and the number of SMs, belong to the device that is current
    first, again, _, other, _, back = run(call, call, "device 1", call, "device 0", call)
    for r in (first, again, other, back):
        assert r["status"] == 0
        (launch,) = r["launches"]
        assert launch["smem"] <= launch["allowed"]
    grids = [r["launches"][0]["grid"] for r in (first, other, back)]
    assert grids[0] == grids[2] and grids[0] % 152 == 0 or "plan" in call and grids[0] == 78
    assert grids[1] % 100 == 0 or "plan" in call and grids[1] == 78


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_a_failed_set_up_is_tried_again(run, call):
    _, failed, after = run("fail 1", call, call)
    assert failed["status"] == 3 and not failed["launches"]
    assert after["status"] == 0 and after["launches"][0]["smem"] <= after["launches"][0]["allowed"]


def test_plan_takes_the_device_it_runs_on(run):
    a, _, b = run("plan 40 1000000", "device 1", "plan 40 1000000")
    assert a["launches"][0]["grid"] == 152 and b["launches"][0]["grid"] == 100


@pytest.mark.parametrize("dt", [BF16, F32])
def test_a_window_that_hides_nothing_changes_nothing(run, dt):
    # 2^31 - 1 keys are more than a request can have
    a, *b = run(*[attention(dt, 1, 6000, 6000, dim=128, width=512, window=w) for w in (0, 2**31 - 129, 2**31 - 128, 2**31 - 1, 2**31)])
    assert all(r["launches"][0]["kernel"] == a["launches"][0]["kernel"] for r in b)
