"""Serving operators for long contexts and drafted tokens at the edges of what
their arguments allow.
"""
import numpy as np
import pytest
import torch

from oracle import context_oracle as co
from test_gpu_context import BF, F, f64, gen, gsi, i32, rotary_case, verify_case  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rotary
@pytest.mark.parametrize("xdt,cdt", [(F, BF), (BF, BF), (F, F), (BF, F)])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,hq,hkv,D,page,n", [(5, 3, 3, 80, 32, 20), (37, 4, 1, 64, 16, 2), (9, 4, 4, 256, 256, 64), (4, 2, 2, 96, 16, 48), (3, 1, 1, 8, 16, 6)])
def test_rotary_copies_what_a_key_has_beside_its_turned_values(gsi, xdt, cdt, layout, T, hq, hkv, D, page, n):  # noqa: F811
    g = gen(T + n)
    rows = torch.randn(T, (hq + 2 * hkv) * D, device="cuda", generator=g).to(xdt)
    cache = gsi.PagedCache(*(torch.zeros(T // page + 1, hkv, page, D, dtype=cdt, device="cuda") for _ in range(2)))
    slots = torch.randperm((T // page + 1) * page, device="cuda", generator=g)[:T]
    slots[T // 2] = -1  # a token that the cache does not get
    gsi.rotary_append(cache, rows, slots, i32(range(1000, 1000 + T)), hq, gsi.Rotary.make(n, 10000.0, layout))
    there = slots >= 0
    got = cache.K[(slots // page).clamp(min=0), :, slots % page][there]
    key = rows.view(T, -1, D)[there, hq:hq + hkv]
    assert torch.equal(got[..., n:], key[..., n:].to(cdt))  # bit for bit
    assert not torch.equal(got[..., :n], key[..., :n].to(cdt))


@pytest.mark.parametrize("xdt,cdt", [(F, BF), (BF, BF), (BF, F)])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,hq,hkv,D,page,n", [(331, 8, 4, 64, 16, 64), (305, 3, 1, 80, 32, 20), (640, 12, 2, 128, 64, 32)])
def test_rotary_of_a_prompt(gsi, xdt, cdt, layout, T, hq, hkv, D, page, n):  # noqa: F811
    # (from twice the SMs on a token has one CTA, whose threads may have several vectors or none)
    rotary_case(gsi, xdt, cdt, T, hq, hkv, D, page, n, layout, list(range(7, 7 + T)))


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("R,hkv,lens,budget,recent,sinks", [
    (30, 8, (16_385, 19_001), 9000, 500, 4),     # 240 heads: a CTA each
    (30, 8, (16_400, 16_393), 16_384, 0, 0),     # few keys given up, more than are looked through one by one
    (15, 8, (32_800, 34_001), 12_345, 64, 64)])  # 120 heads: two CTAs each
def test_evict_more_keys_than_shared_memory_holds_under_many_heads(gsi, R, hkv, lens, budget, recent, sinks):  # noqa: F811
    g = gen(R + budget)
    D, page = 8, 256
    n = [lens[r % 2] - r for r in range(R)]
    width = -(-max(n) // page)
    cache = gsi.PagedCache.empty(R * width, hkv, page, D, BF)
    cache.K.normal_(generator=g), cache.V.normal_(generator=g)
    table = torch.randperm(R * width, device="cuda", generator=g).int().view(R, width)
    # rounded weights: ties, at the border too
    marks = gsi.KeyMarks((torch.randn(R * width, hkv, page, device="cuda", generator=g) * 300).round(),
                         torch.zeros(R * width, hkv, page, dtype=torch.int32, device="cuda"))
    for r in range(R):
        marks.place[table[r].long()] = torch.stack([torch.randperm(width * page, device="cuda", generator=g) for _ in range(hkv)]).int().view(hkv, width, page).transpose(0, 1)
    flat = lambda t: torch.stack([t[table[r].long()].transpose(0, 1).flatten(1, 2) for r in range(R)])  # noqa: E731  (R, hkv, places)
    want = [flat(t).clone() for t in (cache.K, cache.V, marks.weight, marks.place)]
    kept, out = gsi.cache_evict(cache, i32(n), table, marks, budget, recent, sinks)
    assert kept.tolist() == [min(budget, m) for m in n] and out.tolist() == [max(0, m - budget) for m in n]
    for r in range(R):
        if n[r] <= budget:
            continue
        for h in range(hkv):
            w, p = want[2][r, h, :n[r]].clone(), want[3][r, h, :n[r]]
            w[p < sinks] = 1e30
            w[p >= n[r] - recent] = float("inf")
            stay = torch.zeros(n[r], dtype=torch.bool, device="cuda")
            stay[torch.sort(w, descending=True, stable=True).indices[:budget]] = True
            gaps, movers = (~stay[:budget]).nonzero()[:, 0], stay[budget:].nonzero()[:, 0] + budget
            for a in want:
                a[r, h, gaps] = a[r, h, movers]
    for a, b in zip(want, (cache.K, cache.V, marks.weight, marks.place)):
        assert torch.equal(a, flat(b))


# ------------------------------------------------------------------ drafts
@pytest.mark.parametrize("V", [2**18 - 1, 2**18, 2**18 + 1, 300_001])
@pytest.mark.parametrize("tdt,ddt", [(F, F), (BF, BF), (BF, None)])
def test_verify_rows_of_more_mass_than_64_bits_hold(gsi, V, tdt, ddt):  # noqa: F811
    # tokens of 1 each: 2^18 of them are 2^64 of the sums' units, of 2^-46
    def ones(target, draft, tokens, u, v):
        target[:] = 1.0
        u[:] = 1.0  # the certain draft, and the one of 1, do not stand
        if draft is not None:
            draft[:] = 0.0
            draft[:-1].scatter_(1, tokens[1:, None].long(), 1.0)
    got = verify_case(gsi, [0, 1, 2], V, tdt, ddt, seed=V % 7, edit=ones)
    assert got.accepted.tolist() == [0, 0, 0] and got.out[0] >= 0


@pytest.mark.parametrize("R", [1, 400])  # one row over eight CTAs, and in one
def test_verify_the_widest_row(gsi, R):  # noqa: F811
    V, skip = 2**24, 2**20 + 77
    target = torch.ones(1, V, dtype=BF, device="cuda")
    target[0, :skip] = 0.0
    q_start = np.full(R + 1, 0)
    q_start[R:] = 1
    for v in (0.0, 0.3, 0.75, 0.9999, 1 - 2.0**-24):
        samples = torch.full((R,), v, device="cuda")
        got = gsi.verify_drafts(target, None, i32([0]), torch.zeros(1, device="cuda"), samples, i32(q_start))
        # the k-th of equal tokens is the first whose running sum, k + 1, is above v times their number
        assert got.out.tolist() == [skip + int(float(samples[0]) * (V - skip))], v


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("p,q,u,stands", [
    (0.5, NAN, 0.9, True), (0.0, NAN, 0.9, False),     # NaN counts as 0: 0 < p
    (0.5, -0.1, 1.0, True), (0.0, -0.1, 0.5, False),   # so does what is negative
    (-0.1, -0.5, 0.5, False), (NAN, 0.5, 0.0, False), (-0.2, 0.5, 0.0, False),
    (0.95, 2.0, 0.9, True), (0.85, 2.0, 0.9, False),   # above 1 counts as 1
    (INF, 2.0, 0.9, True), (3.0, 2.0, 1.0, False), (3.0, INF, 0.99, True), (1.0, INF, 1.0, False)])
@pytest.mark.parametrize("dt", [F, BF])
def test_verify_takes_a_draft_by_what_its_probabilities_count_as(gsi, p, q, u, stands, dt):  # noqa: F811
    target = torch.tensor([[0.25, p, 0.25, 0.25], [1.0, 0.0, 0.0, 0.0]], device="cuda").to(dt)
    draft = torch.tensor([[0.0, q, 0.0, 0.0], [0.0] * 4], device="cuda").to(dt)
    us, v = torch.tensor([u, 0.0], device="cuda"), torch.tensor([0.999], device="cuda")
    got = gsi.verify_drafts(target, draft, i32([0, 1]), us, v, i32([0, 2]))
    assert got.accepted.tolist() == [int(stands)]
    want = co.verify(f64(target), f64(draft), [0, 1], us.tolist(), v.tolist(), [0, 2])
    assert got.out.tolist() == want[0] and want[1] == [int(stands)]
    if dt is F:  # a certain draft: its 1 against what the target's probability counts as
        got = gsi.verify_drafts(target, None, i32([0, 1]), us, v, i32([0, 2]))
        count = min(max(p, 0.0), 1.0) if p == p else 0.0
        assert got.accepted.tolist() == [int(float(us[0]) < count)]
