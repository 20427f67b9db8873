"""How the attention kernels cut ragged requests into shares, on the CPU.

Every CTA finds its own share of the work from the requests' lengths, in closed
form where it can; a tile that two CTAs take, or none, or a part that is joined
by a CTA that does not hold it, would only show on a GPU.  A C++ harness
(attn_share_dump.cpp) runs the kernels' share arithmetic, blocks and warps
included, and this test compares what the CTAs take with the keys that each
token sees by definition, counted token by token.
"""
import json
import os
import random
import shutil
import subprocess

import pytest

import __graft_entry__

__graft_entry__.build()
from gated_rank_subspace_gb300 import _build  # noqa: E402
from oracle.serving_oracle import keys_of  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))
# kernel: threads, query rows of a unit, keys of a tile, tiles that a unit counts beside its own
KERNELS = {"rows, 128 keys": (384, 8, 128, 0), "rows, 64 keys": (384, 8, 64, 0), "two row tiles": (384, 256, 128, 2),
           "one row tile": (256, 128, 128, 2), "float32": (256, 64, 64, 0), "float32, few rows": (256, 16, 64, 0)}


def unit_tokens(kernel, group):
    rows = KERNELS[kernel][1]
    return 2 * (128 // group) if rows == 256 else rows // group


def line(kernel, grid, hkv, group, causal, window, page_shift, width, lens, first=0, N=None):
    nt, _, kt, extra = KERNELS[kernel]
    start = [first]
    for q, _ in lens:
        start.append(start[-1] + q)
    N = start[-1] if N is None else N
    return " ".join(map(str, [nt, grid, unit_tokens(kernel, group), kt, extra, hkv, group, causal, window, page_shift, width, N, len(lens),
                              *start, *(k for _, k in lens)]))


def cases():
    out = []
    rng = random.Random(3)
    for kernel, (_, rows, kt, _) in KERNELS.items():
        groups = [g for g in (1, 2, 3, 4, 6, 7, 8, 12, 16, 50, 64, 128) if g <= min(rows, 128)]
        for i in range(36):
            group, hkv, grid = rng.choice(groups), rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 5, 9, 16])
            n_req, causal = rng.choice([1, 1, 2, 3, 9, 40]), rng.random() < 0.8
            window = rng.choice([0, 0, 1, 17, 128, 300, 5000]) if causal else 0
            most_q, most_k = rng.choice([(1, 900), (3, 60), (40, 700), (700, 2000), (300, 100)])
            if n_req == 40:
                most_q, most_k = min(most_q, 5), min(most_k, 300)
            lens = [(rng.randint(0, most_q), rng.randint(0, most_k)) for _ in range(n_req)]
            if i % 4 == 0:  # a prompt alone: as many keys as tokens, or some more
                q = rng.randint(1, 3000 if rows > 16 else 90)
                lens, causal, window = [(q, q + rng.choice([0, 0, 1, 500]))], True, 0
            lens[rng.randrange(n_req if len(lens) == n_req else 1)] = rng.choice(lens)
            out.append((kernel, grid, hkv, group, int(causal), window, 6, 1 + max(k for _, k in lens) // 64, lens))
        # whole grids
        for grid in (152, 2 * 152) if kt == 64 and KERNELS[kernel][0] == 256 else (152,):
            out.append((kernel, grid, 4, 1, 1, 0, 4, 600, [(rng.randint(0, 30), rng.randint(0, 9000)) for _ in range(5)]))
            out.append((kernel, grid, 16, 1, 1, 0, 4, 130, [(min(2048, 24 * rows), 2048)]))
        if KERNELS[kernel][3]:  # units of many tiles, cut several times, some of the cuts near their ends
            for _ in range(30):
                lens = [(rng.randint(30, 400), rng.randint(2000, 12000)) for _ in range(rng.choice([2, 3]))]
                out.append((kernel, rng.choice([16, 31, 40]), rng.choice([1, 2, 3]), rng.choice([1, 2, 4]), rng.choice([0, 1]), 0, 6, 200, lens))
    # more keys than the table holds
    out.append(("one row tile", 7, 2, 4, 1, 0, 4, 10, [(200, 500), (50, 160), (3, 161)]))
    return out


@pytest.fixture(scope="module")
def dump(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not available")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    exe = str(tmp_path_factory.mktemp("share") / "attn_share_dump")
    subprocess.run([gxx, "-std=c++17", "-O2", "-I", _build.INCLUDE, "-I", _build.CSRC, "-I", os.path.join(cuda, "include"),
                    os.path.join(HERE, "attn_share_dump.cpp"), "-o", exe], check=True)

    def go(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [json.loads(x) for x in r.stdout.splitlines()]

    return go


def units_of(kernel, hkv, group, causal, window, page, width, lens):
    """Every unit (request, head, block of tokens) and its tiles [t0, t0 + n), from the keys of each token."""
    ut, kt = unit_tokens(kernel, group), KERNELS[kernel][2]
    out = {}
    for r, (q, k) in enumerate(lens):
        k = min(k, width * page)
        for u in range(-(-q // ut)):
            seen = [keys_of(q, k, i, causal, window) for i in range(u * ut, min(q, (u + 1) * ut))]
            seen = [(lo, lim) for lo, lim in seen if lim > lo]
            t0 = min((lo for lo, _ in seen), default=0) // kt
            t1 = -(-max((lim for _, lim in seen), default=0) // kt)
            for h in range(hkv):
                out[r, h, u] = (t0, t1 - t0)
    return out


def check(got, kernel, grid, hkv, group, causal, window, page_shift, width, lens):
    assert got["alike"], "the threads of a block disagree"
    units = units_of(kernel, hkv, group, causal, window, 1 << page_shift, width, lens)
    parts = {}
    for cta, segments in enumerate(got["ctas"]):
        begun = ended = 0
        for r, h, u, t0, n, a, b, b0, b1 in segments:
            want_t0, want_n = units[r, h, u]
            assert n == want_n and (n == 0 or t0 == want_t0)
            assert 0 <= a <= b <= n
            parts.setdefault((r, h, u), []).append((cta, a, b, b0, b1))
            if not (a == 0 and b == n):  # a part: it has one of the CTA's two places in the workspace
                begun, ended = begun + (b0 == cta), ended + (b0 != cta)
        assert begun <= 1 and ended <= 1, "two parts in one place"
    assert parts.keys() == units.keys(), "a unit that no CTA takes"
    for unit, (_, n) in units.items():
        held = parts[unit]
        if any(a == 0 and b == n for _, a, b, _, _ in held):
            assert len(held) == 1 or n == 0, "a whole unit and another part of it"
            continue
        assert got["dealt"] == 0
        ctas, b0, b1 = [p[0] for p in held], held[0][3], held[0][4]
        assert ctas == list(range(b0, b1 + 1)) and all(p[3:] == (b0, b1) for p in held), "the CTAs that join a unit are others"
        assert [p[1] for p in held] == [0] + [p[2] for p in held[:-1]] and held[-1][2] == n, "a tile twice, or never"
    # equal shares: to a tile where units count for nothing more, and within what moved cuts change otherwise
    if got["dealt"] == 0 and units:
        tiles = [sum(max(s[6] - s[5], s[4] == 0) for s in c) for c in got["ctas"]]
        most = -(-got["total"] // got["grid"])
        assert max(tiles) <= most + 2 * got["extra"]
        if not got["extra"]:
            assert sum(tiles) == got["total"] and most == -(-got["total"] // min(grid, got["total"])), "a longer share than need be"


@pytest.fixture(scope="module")
def results(dump):
    all_cases = cases()
    return list(zip(all_cases, dump([line(*c) for c in all_cases]), strict=True))


def test_every_tile_is_taken_once_and_joined_by_those_who_hold_it(results):
    for case, got in results:
        try:
            check(got, *case)
        except AssertionError as e:
            raise AssertionError(f"{case}: {e}") from e


def test_the_cases_reach_every_way_to_cut(results):
    got = [g for _, g in results]
    assert any(g["dealt"] for g in got) and any(g["extra"] for g in got)
    assert any(not g["extra"] and not g["dealt"] for g in got)
    assert any(b1 - b0 > 3 for g in got if not g["dealt"] for c in g["ctas"] for *_, b0, b1 in c)


def test_tokens_outside_every_request_and_lengths_out_of_range(dump):
    # padding before the first token and behind the last; a request that says it has more than there are
    g, = dump([line("rows, 128 keys", 5, 2, 1, 1, 0, 4, 20, [(8, 300), (0, 9), (9, 9)], first=3, N=40)])
    check(g, "rows, 128 keys", 5, 2, 1, 1, 0, 4, 20, [(8, 300), (0, 9), (9, 9)])
    g, = dump([line("rows, 128 keys", 5, 2, 1, 1, 0, 4, 20, [(8, 300), (9, -4)], N=12)])
    check(g, "rows, 128 keys", 5, 2, 1, 1, 0, 4, 20, [(8, 300), (4, 0)])


def test_no_work_is_no_share(dump):
    g, = dump([line("float32", 5, 2, 1, 1, 0, 4, 20, [(0, 300), (0, 0)])])
    assert all(c == [] for c in g["ctas"]) and g["alike"]
