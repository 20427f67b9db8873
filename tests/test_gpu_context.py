"""Serving operators for long contexts and drafted tokens on the GPU against
their float64 definitions.

Tolerances, from the arithmetic the kernels do:
  * rotary: an angle is known to 2^-32 of a turn, its float32 sine and cosine to
    2 ulp, and two products are rounded: |error| <= scale (|a| + |b|) 2^-21 for
    the pair (a, b); a bf16 result adds half a step, 2^-8 of it.  What is not
    turned is a copy, or one rounding: equal bit for bit;
  * the logarithm of a row's sum: scores of magnitude <= ~20 from up to 256
    float32 products (2e-5 of absolute error, as for the attention); bf16 sums the
    weights as they were rounded, each by up to 2^-8: ln(1 + 2^-8) < 2^-8; and the
    float32 logarithm's own 2^-22 of its magnitude;
  * gathered weights: exp(x) has the relative error of x's absolute one: 2e-5 as
    above, doubled for the products' order, and 2^-24 of the sum for each of up to
    2^7 additions in a row: 1e-4 of what is gathered covers it twice;
  * eviction, verification, pages: whole numbers and copies, equal.
"""
import numpy as np
import pytest
import torch

from oracle import context_oracle as co

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gsi():
    import __graft_entry__
    __graft_entry__.build()
    import gated_rank_subspace_gb300 as g
    assert torch.cuda.is_available()
    return g


def i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ rotary
def rotary_case(gsi, xdt, cdt, T, hq, hkv, D, page, n, layout, positions, scale=1.25, offsets=None, req=None, pad=8):
    g = gen(T + D)
    width = (hq + 2 * hkv) * D
    wide = torch.randn(T, width + 2 * pad, device="cuda", generator=g).to(xdt)
    rows = wide[:, pad:pad + width]
    pages = 2 * -(-T // page) + 1
    cache = gsi.PagedCache.empty(pages, hkv, page, D, cdt)
    cache.K.normal_(generator=g), cache.V.normal_(generator=g)
    K, V = cache.K.clone(), cache.V.clone()
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:T]
    if T > 2:
        slots[T // 2] = -1
    turn = gsi.Rotary.make(n, 10000.0, layout)
    turn.scale = scale
    got = gsi.rotary_append(cache, rows, slots, i32(positions), hq, turn, token_req=None if req is None else i32(req),
                            offsets=None if offsets is None else i32(offsets))
    p = np.asarray(positions, dtype=np.int64)
    if offsets is not None:
        p = p + np.array([offsets[q] if 0 <= q < len(offsets) else 0 for q in (req if req is not None else [0] * T)])
    x = f64(rows).reshape(T, -1, D)
    want = co.rotary(x[:, :hq + hkv], p, co.Angle(turn.phases.tolist()), layout, scale)
    size = np.abs(x[:, :hq + hkv])
    if layout == "half":
        pair = size[..., :n // 2] + size[..., n // 2:n]
        pair = np.concatenate([pair, pair], -1)
    else:
        pair = np.repeat(size[..., 0:n:2] + size[..., 1:n:2], 2, -1)
    tol = scale * pair * 2**-21 + (np.abs(want[..., :n]) * 2**-8 if cdt is BF else 0)

    def same(out, lo, hi):
        assert (np.abs(out[..., :n] - want[:, lo:hi, :n]) <= tol[:, lo:hi]).all(), np.abs(out[..., :n] - want[:, lo:hi, :n]).max()
        copy = rows.reshape(T, -1, D)[:, lo:hi, n:].to(cdt)
        assert np.array_equal(out[..., n:], f64(copy))

    same(f64(got), 0, hq)
    ok = (slots >= 0).cpu().numpy()
    pg, off = (slots // page).clamp(min=0), slots % page
    k = f64(cache.K[pg, :, off])
    k[~ok] = want[~ok][:, hq:]  # not written
    if ok.all():
        same(k, hq, hq + hkv)
    else:
        assert (np.abs(k[..., :n] - want[:, hq:, :n]) <= tol[:, hq:]).all()
    assert torch.equal(cache.V[pg, :, off][slots >= 0], rows.reshape(T, -1, D)[:, hq + hkv:].to(cdt)[slots >= 0])
    keep = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    keep[slots[slots >= 0]] = False
    flat = lambda t: t.transpose(1, 2).reshape(pages * page, hkv, D)  # noqa: E731
    assert torch.equal(flat(cache.K)[keep], flat(K)[keep]) and torch.equal(flat(cache.V)[keep], flat(V)[keep])


@pytest.mark.parametrize("xdt,cdt", [(F, BF), (BF, BF), (F, F), (BF, F)])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,hq,hkv,D,page,n", [(1, 8, 2, 128, 16, 128), (5, 3, 3, 80, 32, 20), (37, 4, 1, 64, 16, 2), (3, 0, 2, 16, 64, 16),
                                               (9, 4, 4, 256, 256, 64), (4, 2, 2, 96, 16, 48), (2, 16, 16, 256, 16, 256), (3, 1, 1, 8, 16, 6)])
def test_rotary_append(gsi, xdt, cdt, layout, T, hq, hkv, D, page, n):
    rotary_case(gsi, xdt, cdt, T, hq, hkv, D, page, n, layout, list(range(1000, 1000 + T)))


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rotary_far_and_moved_positions(gsi, layout):
    far = [0, 1, -1, 2**31 - 1, -2**31, 10**6 + 1, 7, 8]
    rotary_case(gsi, F, F, 8, 2, 1, 64, 16, 64, layout, far)
    rotary_case(gsi, F, BF, 8, 2, 1, 64, 16, 32, layout, far, offsets=[5, -3, 2**31 - 1], req=[0, 1, 2, 2, 1, -1, 3, 0])
    rotary_case(gsi, F, F, 2, 2, 1, 64, 16, 32, layout, [4, 5], offsets=[77])


def test_rotary_of_zero_angle_is_the_append(gsi):
    rows = torch.randn(5, 4 * 64, device="cuda", generator=gen(0))
    a, b = (gsi.PagedCache(*(torch.zeros(2, 1, 16, 64, dtype=BF, device="cuda") for _ in range(2))) for _ in range(2))
    slots = torch.arange(5, device="cuda")
    q = gsi.cache_append(a, rows, slots, 2)
    p = gsi.rotary_append(b, rows, slots, i32([0] * 5), 2, gsi.Rotary.make(64))
    assert torch.equal(p, q) and torch.equal(a.K, b.K) and torch.equal(a.V, b.V)
    q = gsi.rotary_append(b, rows[:0], slots[:0], i32([]), 2, gsi.Rotary.make(64))
    assert q.shape == (0, 2, 64) and torch.equal(a.K, b.K)


def test_rotary_in_a_permuted_cache(gsi):
    buf = [torch.zeros(3, 16, 2, 64, dtype=BF, device="cuda") for _ in range(2)]
    a = gsi.PagedCache(*(t.permute(0, 2, 1, 3) for t in buf))
    b = gsi.PagedCache(*(torch.zeros(3, 2, 16, 64, dtype=BF, device="cuda") for _ in range(2)))
    rows = torch.randn(20, 6 * 64, device="cuda", generator=gen(1))
    slots, pos = torch.randperm(48, device="cuda", generator=gen(2))[:20], i32(range(20))
    for c in (a, b):
        gsi.rotary_append(c, rows, slots, pos, 2, gsi.Rotary.make(32, layout="pairs"))
    assert torch.equal(a.K, b.K) and torch.equal(a.V, b.V)


# ------------------------------------------------------------------ weights of keys
def paged(lens, page, extra, g, width=None):
    want = [-(-n // page) for n in lens]
    pages = sum(want) + extra
    ids = torch.randperm(pages, device="cuda", generator=g).int().cpu().numpy()
    table = np.full((len(lens), width or max([1] + want)), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(want):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, pages


class Weights:
    def __init__(self, gsi, dt, hq, hkv, D, page, lens, seed=0, held=None, offsets=None, causal=True, scale=None, stride=0):
        g = gen(seed + D)
        self.gsi, self.causal, self.scale = gsi, causal, D**-0.5 if scale is None else scale
        self.table, pages = paged([n for _, n in lens], page, 2, g)
        self.cache = gsi.PagedCache.empty(pages, hkv, page, D, dt)
        self.cache.K.normal_(generator=g), self.cache.V.normal_(generator=g)
        N = sum(q for q, _ in lens)
        wide = torch.randn(N, hq * D + stride, device="cuda", generator=g).mul_(2).to(dt)
        self.Q = wide[:, :hq * D].view(N, hq, D) if not stride else wide.as_strided((N, hq, D), (hq * D + stride, D, 1))
        self.q_start = np.concatenate([[0], np.cumsum([q for q, _ in lens])])
        self.kv_len = [n for _, n in lens]
        self.held, self.offsets = held, offsets
        self.marks = gsi.KeyMarks(torch.rand(pages, hkv, page, device="cuda", generator=g),
                                  torch.randint(0, 99, (pages, hkv, page), device="cuda", generator=g).int())
        L = co.lse(f64(self.Q), f64(self.cache.K), self.q_start, self.kv_len, self.table, self.scale, causal)
        self.lse = torch.tensor(L, device="cuda").float()

    def run(self, max_q=None, **kw):
        m = self.gsi.KeyMarks(self.marks.weight.clone(), self.marks.place.clone())
        opt = lambda v: None if v is None else i32(v)  # noqa: E731
        self.gsi.key_weights(self.cache, self.Q, self.lse, i32(self.q_start), i32(self.kv_len), i32(self.table), m,
                             held=opt(self.held), offsets=opt(self.offsets), max_q=max_q, scale=self.scale, causal=self.causal, **kw)
        return m

    def check(self, max_q=None):
        got = self.run(max_q)
        w, p = co.key_weights(f64(self.Q), f64(self.cache.K), f64(self.lse), self.q_start, self.kv_len, self.held, self.offsets,
                              self.table, f64(self.marks.weight), self.marks.place.cpu().numpy(), self.scale, self.causal)
        assert np.array_equal(got.place.cpu().numpy(), p)
        g = f64(got.weight)
        assert np.array_equal(np.isnan(g), np.isnan(w))
        far = np.abs(g - w)[np.isfinite(w)] - 1e-4 * np.abs(w)[np.isfinite(w)]
        assert (far <= 1e-30).all(), (far.max(), np.abs(g - w).max())
        return got


LENS = [[(1, 1)], [(1, 77), (1, 3)], [(3, 200), (1, 1), (0, 40)], [(70, 300)], [(130, 130), (1, 129), (5, 5)], [(40, 9), (2, 64)],
        [(0, 5)], [(1, 700), (33, 513), (0, 0), (2, 128)]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dt,hq,hkv,D,page", [(BF, 2, 2, 128, 16), (BF, 8, 2, 64, 32), (BF, 2, 2, 256, 64), (BF, 3, 1, 80, 256),
                                              (BF, 6, 2, 192, 128), (F, 2, 2, 64, 16), (F, 6, 2, 20, 32)])
def test_key_weights(gsi, lens, dt, hq, hkv, D, page):
    Weights(gsi, dt, hq, hkv, D, page, lens).check(max_q=max(1, max(q for q, _ in lens)))


@pytest.mark.parametrize("dt,D", [(BF, 8), (BF, 16), (BF, 40), (BF, 136), (F, 4), (F, 100), (F, 252)])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 3)], [(3, 200), (1, 1)], [(70, 300)]], ids=str)
def test_key_weights_odd_head_sizes(gsi, dt, D, lens):
    Weights(gsi, dt, 4, 2, D, 32, lens).check(max(q for q, _ in lens))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 16)])
def test_key_weights_of_units_of_one_and_more_steps(gsi, D, page):
    # a few-row kernel's units of one, two and five steps in turn: the warpgroups change places, and whose turn a place in the
    # rings is
    lens = [(1, 500), (20, 400), (1, 900), (33, 300), (1, 130), (70, 200)] * 4
    w = Weights(gsi, BF, 2, 2, D, page, lens, held=[max(0, n - q) for q, n in lens])
    ref = w.check(1)
    for _ in range(3):
        assert torch.equal(w.run(1).weight, ref.weight)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 3)], [(20, 300), (0, 200), (1, 130)], [(130, 260)]], ids=str)
def test_key_weights_gathered_over_steps(gsi, dt, lens):
    held = [max(0, n - q) for q, n in lens]
    held[-1] = lens[-1][1] // 2  # more keys are new than have a row here
    w = Weights(gsi, dt, 4, 2, 64, 16, lens, held=held, offsets=[7 * i for i in range(len(lens))])
    w.check()
    w.held = [n + 5 for _, n in lens]  # every key had marks
    w.check()


@pytest.mark.parametrize("dt,group", [(BF, 1), (BF, 5), (BF, 16), (BF, 17), (BF, 64), (BF, 65), (BF, 128), (F, 5), (F, 64), (F, 65), (F, 128)])
@pytest.mark.parametrize("max_q", [0, 1, 1000])
def test_key_weights_of_shared_heads_and_any_hint(gsi, dt, group, max_q):
    Weights(gsi, dt, group, 1, 32, 16, [(3, 150), (1, 200), (9, 9)]).check(max_q)


@pytest.mark.parametrize("dt", [BF, F])
def test_key_weights_of_cross_attention_layout_and_scale(gsi, dt):
    Weights(gsi, dt, 4, 2, 64, 16, [(20, 9), (150, 300), (3, 0)], causal=False).check()
    Weights(gsi, dt, 4, 2, 64, 16, [(20, 90), (1, 300)], scale=-0.05, stride=64).check()
    Weights(gsi, dt, 4, 2, 64, 16, [(20, 90), (1, 300)], scale=0.0).check()
    w = Weights(gsi, dt, 4, 2, 64, 16, [(20, 90), (1, 300)])
    ref = w.run().weight
    K = w.cache.K.transpose(1, 2).contiguous().transpose(1, 2)
    w.cache = gsi.PagedCache(K, K)
    assert torch.equal(w.run().weight, ref)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("lens", [[(1, 40), (1, 200)], [(140, 300)]], ids=str)
def test_key_weights_table_entries_outside_the_cache(gsi, dt, lens):
    w = Weights(gsi, dt, 4, 2, 64, 16, lens)
    w.table[0, 1], w.table[-1, 0] = -5, 10**6
    w.check()


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_key_weights_nonfinite_keys_stay_with_their_key(gsi, dt, value):
    w = Weights(gsi, dt, 4, 2, 64, 16, [(1, 40), (130, 200)])
    place = int(w.table[0, 1])
    w.cache.K[place, :, 3] = value  # key 19 of request 0
    stale = int(w.table[1, -1])
    w.cache.K[stale, :, 8:] = value  # behind the last key of request 1
    got, ref = w.run(), Weights(gsi, dt, 4, 2, 64, 16, [(1, 40), (130, 200)]).run()  # (the logarithms are of the keys as they were)
    if value != value:
        assert got.weight[place, :, 3].isnan().all()
    keep = torch.ones_like(got.weight, dtype=torch.bool)
    keep[place, :, 3] = False
    assert torch.equal(got.weight[keep], ref.weight[keep])


@pytest.mark.parametrize("dt", [BF, F])
def test_key_weights_rows_without_a_sum(gsi, dt):
    # rows that see no key give nothing, whatever their logarithm says
    w = Weights(gsi, dt, 4, 2, 64, 16, [(40, 9)])
    w.lse[:31] = float("nan")
    w.check()


@pytest.mark.parametrize("dt,D,hq,hkv,lens", [(BF, 128, 8, 8, [(1, 3000), (1, 9000)]), (BF, 128, 32, 32, [(1, 8000)] * 6), (BF, 256, 16, 16, [(1, 6000)] * 4), (BF, 64, 8, 1, [(600, 600)]), (BF, 256, 4, 4, [(500, 1200)]),
                                              (F, 64, 4, 4, [(300, 700), (1, 2000)])])
def test_key_weights_long(gsi, dt, D, hq, hkv, lens):
    g = gen(D)
    table, pages = paged([n for _, n in lens], 32, 3, g)
    cache = gsi.PagedCache.empty(pages, hkv, 32, D, dt)
    cache.K.normal_(generator=g), cache.V.normal_(generator=g)
    N = sum(q for q, _ in lens)
    Q = torch.randn(N, hq, D, device="cuda", generator=g).to(dt)
    qs, kv, tab = i32(np.concatenate([[0], np.cumsum([q for q, _ in lens])])), i32([n for _, n in lens]), i32(table)
    lse = torch.empty(N, hq, device="cuda")
    gsi.paged_attention(cache, Q, qs, kv, tab, max_q=max(q for q, _ in lens), lse=lse)
    marks = gsi.KeyMarks.empty(cache)
    marks.weight.fill_(-1)
    again = gsi.KeyMarks(marks.weight.clone(), marks.place.clone())
    work = gsi.new_workspace(gsi.key_weights_workspace_size())
    gsi.key_weights(cache, Q, lse, qs, kv, tab, marks, max_q=max(q for q, _ in lens), workspace=work)
    gsi.key_weights(cache, Q, lse, qs, kv, tab, again, max_q=max(q for q, _ in lens), workspace=work)
    assert torch.equal(marks.weight, again.weight) and gsi.workspace_status(work) == 0
    assert not work.any() or not work[256:256 + 4096].any()  # the counters are back at zero
    a = 0
    for r, (q, n) in enumerate(lens):
        at = tab[r, :-(-n // 32)].long()
        seen = torch.arange(n, device="cuda") <= torch.arange(q, device="cuda")[:, None] + n - q
        got = marks.weight[at].transpose(0, 1).reshape(hkv, -1)[:, :n].double()
        assert torch.equal(marks.place[at].transpose(0, 1).reshape(hkv, -1)[:, :n], torch.arange(n, device="cuda").int().expand(hkv, -1))
        for h in range(hkv):
            k = cache.K[at, h].reshape(-1, D)[:n].double()
            want = torch.zeros(n, dtype=torch.float64, device="cuda")
            for x in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                s = (Q[a:a + q, x].double() @ k.T) * D**-0.5 - lse[a:a + q, x, None].double()
                want += torch.where(seen, s.exp(), 0.0).sum(0)
            assert ((got[h] - want).abs() <= 1e-4 * want).all()
            # what all rows give is one each, but for the rounding of the weights that were summed
            assert abs(want.sum().item() - q * (hq // hkv)) <= 2**-8 * q * (hq // hkv)
        a += q


@pytest.mark.parametrize("dt,hq,hkv", [(BF, 2, 1), (F, 2, 1)])
def test_key_weights_of_many_requests(gsi, dt, hq, hkv):
    rng = np.random.default_rng(3)
    lens = [(int(q), int(q + n)) for q, n in zip(rng.integers(0, 3, 700), rng.integers(0, 40, 700))]
    Weights(gsi, dt, hq, hkv, 32, 16, lens, held=[max(0, n - q) for q, n in lens], offsets=rng.integers(0, 9, 700).tolist()).check(2)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("lens", [[(1, 700), (1, 20)], [(40, 300), (200, 260)]], ids=str)
def test_key_weights_on_another_stream_and_in_graphs(gsi, dt, lens):
    """One workspace for the attention, the weights and the eviction, in two graphs of a stream, replayed in turn."""
    w = Weights(gsi, dt, 4, 2, 64, 16, lens)
    ref = w.run().weight
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w.run(stream=s)
    s.synchronize()
    assert torch.equal(got.weight, ref)
    N, hq = w.Q.shape[:2]
    ws = gsi.new_workspace(max(gsi.paged_attention_workspace_size(w.cache, hq), gsi.key_weights_workspace_size(),
                               gsi.cache_evict_workspace_size(w.cache, len(lens), 16)))
    args = (i32(w.q_start), i32(w.kv_len), i32(w.table))
    out, lse = torch.empty_like(w.Q), torch.empty(N, hq, device="cuda")
    a, b = (gsi.KeyMarks(w.marks.weight.clone(), w.marks.place.clone()) for _ in range(2))
    kept, gone = torch.empty_like(args[1]), torch.empty_like(args[1])
    want = gsi.paged_attention(w.cache, w.Q, *args)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        gsi.paged_attention(w.cache, w.Q, *args, out=out, lse=lse, workspace=ws)
        gsi.key_weights(w.cache, w.Q, w.lse, *args, a, workspace=ws)
    scratch = gsi.PagedCache(w.cache.K.clone(), w.cache.V.clone())
    with torch.cuda.graph(second):
        gsi.key_weights(w.cache, w.Q, w.lse, *args, b, workspace=ws)
        gsi.cache_evict(scratch, args[1], args[2], gsi.KeyMarks(b.weight, b.place), 16, kept=kept, offsets_out=gone, workspace=ws)
    keep = None
    for _ in range(3):
        a.weight.zero_(), b.weight.zero_(), out.zero_()
        scratch.K.copy_(w.cache.K), scratch.V.copy_(w.cache.V)
        first.replay(), second.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        table, valid = args[2].long(), [n for _, n in lens]
        for r, n in enumerate(valid):
            pg = table[r, torch.arange(n, device="cuda") // 16]
            assert torch.equal(a.weight[pg, :, torch.arange(n, device="cuda") % 16], ref[pg, :, torch.arange(n, device="cuda") % 16])
        assert kept.tolist() == [min(16, n) for n in valid]
        now = (scratch.K.clone(), b.weight.clone(), b.place.clone())
        assert keep is None or all(torch.equal(x, y) for x, y in zip(keep, now))
        keep = now
    assert gsi.workspace_status(ws) == 0


# ------------------------------------------------------------------ the attention's logarithms
@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 500), (1, 3)], [(3, 200), (0, 7), (1, 1)], [(150, 400), (40, 9)], [(1, 5000)], [(300, 900)]], ids=str)
@pytest.mark.parametrize("dt,hq,hkv,D", [(BF, 2, 2, 128), (BF, 16, 2, 64), (BF, 2, 2, 256), (F, 4, 2, 64), (F, 70, 1, 32)])
@pytest.mark.parametrize("window", [0, 100])
def test_attention_lse(gsi, lens, dt, hq, hkv, D, window):
    w = Weights(gsi, dt, hq, hkv, D, 16, lens)
    args = (w.cache, w.Q, i32(w.q_start), i32(w.kv_len), i32(w.table))
    kw = dict(max_q=max(q for q, _ in lens), window=window)
    got = torch.full((w.Q.shape[0] , hq), 5.0, device="cuda")
    O = gsi.paged_attention(*args, lse=got, **kw)
    assert torch.equal(O, gsi.paged_attention(*args, **kw))
    want = co.lse(f64(w.Q), f64(w.cache.K), w.q_start, w.kv_len, w.table, w.scale, True, window)
    g = f64(got)
    assert np.array_equal(np.isinf(g), np.isinf(want))
    ok = np.isfinite(want)
    tol = 2e-5 + (2**-8 if dt is BF else 0) + np.abs(want[ok]) * 2**-22
    assert (np.abs(g[ok] - want[ok]) <= tol).all(), np.abs(g[ok] - want[ok]).max()


# ------------------------------------------------------------------ eviction
def evict_case(gsi, dt, hkv, D, page, lens, budget, recent=0, sinks=0, offsets=None, seed=0, edit=None, weights=None, extra=2):
    g = gen(seed + D)
    table, pages = paged(lens, page, extra, g)
    cache = gsi.PagedCache.empty(pages, hkv, page, D, dt)
    cache.K.normal_(generator=g), cache.V.normal_(generator=g)
    marks = gsi.KeyMarks(torch.randn(pages, hkv, page, device="cuda", generator=g), torch.zeros(pages, hkv, page, dtype=torch.int32, device="cuda"))
    if weights is not None:
        marks.weight.copy_(weights(marks.weight))
    off = [0] * len(lens) if offsets is None else offsets
    rng = np.random.default_rng(seed)
    for r, n in enumerate(lens):
        for h in range(hkv):
            order = torch.tensor(rng.permutation(n + off[r])[:n].astype(np.int32), device="cuda")
            j = torch.arange(n, device="cuda")
            marks.place[i32(table[r])[j // page].long(), h, j % page] = order
    if edit:
        edit(table, cache, marks)
    before = [f64(cache.K), f64(cache.V), f64(marks.weight), marks.place.cpu().numpy()]
    kept, out = gsi.cache_evict(cache, i32(lens), i32(table), marks, budget, recent, sinks, None if offsets is None else i32(offsets))
    want = co.evict(before[0], before[1], lens, table, before[2], before[3], budget, recent, sinks, offsets)
    for g_, w_, name in zip((f64(cache.K), f64(cache.V), f64(marks.weight), marks.place.cpu().numpy(), kept.tolist(), out.tolist()), want,
                            ("K", "V", "weight", "place", "kept", "offsets")):
        assert np.array_equal(np.asarray(g_), np.asarray(w_), equal_nan=name in ("K", "V", "weight")), name
    return cache, marks


@pytest.mark.parametrize("dt,hkv,D,page", [(BF, 2, 64, 16), (F, 3, 20, 32), (BF, 1, 256, 256), (F, 1, 256, 64), (BF, 4, 8, 16)])
@pytest.mark.parametrize("lens,budget,recent,sinks", [([1], 1, 0, 0), ([2], 1, 0, 0), ([33, 32, 31], 32, 0, 0), ([100, 7, 300, 0], 50, 10, 3),
                                                      ([600], 599, 0, 4), ([600], 1, 1, 0), ([257, 513], 256, 200, 56), ([40] * 9, 17, 0, 0)])
def test_evict(gsi, dt, hkv, D, page, lens, budget, recent, sinks):
    evict_case(gsi, dt, hkv, D, page, lens, budget, recent, sinks)
    evict_case(gsi, dt, hkv, D, page, lens, budget, recent, sinks, offsets=[3 * r for r in range(len(lens))], seed=1)


@pytest.mark.parametrize("weights", [lambda w: w * 0, lambda w: (w * 2).round() / 8, lambda w: w.abs() * 1e-40, lambda w: w * 0 - 0.0,
                                     lambda w: 1 + (w * 4).round() * 2**-23, lambda w: torch.where(w > 1, float("nan"), w),
                                     lambda w: torch.where(w > 0.5, float("inf"), torch.where(w < -1, -float("inf"), w))],
                         ids=["zero", "ties", "subnormal", "negative zero", "last bits", "nan", "inf"])
@pytest.mark.parametrize("budget", [1, 100, 150, 199])
def test_evict_by_any_weights(gsi, weights, budget):
    evict_case(gsi, BF, 2, 16, 16, [200, 200], budget, weights=weights)


@pytest.mark.parametrize("R,hkv,n,budget", [(1, 1, 5000, 1300), (1, 2, 5000, 4999), (40, 2, 700, 350), (5, 1, 3000, 10), (160, 1, 100, 64)])
def test_evict_over_any_number_of_blocks(gsi, R, hkv, n, budget):
    evict_case(gsi, BF, hkv, 8, 64, [max(1, n - 37 * (r % 5)) for r in range(R)], budget, recent=budget // 8, sinks=2)


def test_evict_more_keys_than_shared_memory_holds(gsi):
    n, budget = 150_000, 70_001
    g = gen(3)
    pages = -(-n // 256)
    cache = gsi.PagedCache.empty(pages, 1, 256, 8, BF)
    cache.K.normal_(generator=g), cache.V.normal_(generator=g)
    table = torch.randperm(pages, device="cuda", generator=g).int()[None]
    marks = gsi.KeyMarks((torch.randn(pages, 1, 256, device="cuda", generator=g) * 500).round(), torch.arange(pages * 256, device="cuda").int().view(pages, 1, 256))
    flat = lambda t: t[table[0].long(), 0].flatten(0, 1)[:n].clone()  # noqa: E731
    K, V, w, p = (flat(t) for t in (cache.K, cache.V, marks.weight, marks.place))
    kept, out = gsi.cache_evict(cache, i32([n]), table, marks, budget)
    assert kept.item() == budget and out.item() == n - budget
    stay = torch.zeros(n, dtype=torch.bool, device="cuda")
    # (places are numbers of the cache here: those from n on count as the last positions)
    stay[torch.sort(torch.where(p >= n, float("inf"), w), descending=True, stable=True).indices[:budget]] = True
    gaps, movers = (~stay[:budget]).nonzero()[:, 0], stay[budget:].nonzero()[:, 0] + budget
    for a, b in zip((K, V, w, p), (cache.K, cache.V, marks.weight, marks.place)):
        a[gaps] = a[movers]
        assert torch.equal(a, flat(b))


def test_evict_with_table_entries_outside_the_cache(gsi):
    def edit(table, cache, marks):
        table[0, 0], table[0, 5], table[1, 3] = -1, 10**6, -7
    evict_case(gsi, BF, 2, 16, 16, [200, 100], 40, 5, 2, edit=edit)


def test_evict_in_a_permuted_cache(gsi):
    lens, hkv, D, page = [200, 90, 30], 3, 40, 16
    table, pages = paged(lens, page, 1, gen(1))
    K, V = (torch.randn(pages, hkv, page, D, device="cuda", generator=gen(2)).to(BF) for _ in range(2))
    W, P = torch.randn(pages, hkv, page, device="cuda", generator=gen(3)), torch.arange(pages * hkv * page, device="cuda").int().view(pages, hkv, page)
    got = []
    for layout in (lambda t: t.clone(), lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)):
        for budget in (50, 199):
            cache, marks = gsi.PagedCache(layout(K), layout(V)), gsi.KeyMarks(W.clone(), P.clone())
            gsi.cache_evict(cache, i32(lens), i32(table), marks, budget)
            got.append((cache.K, cache.V, marks.weight, marks.place))
    assert all(torch.equal(a, b) for i in (0, 1) for a, b in zip(got[i], got[i + 2]))


def test_evict_keeps_the_last_and_first_positions(gsi):
    n, budget = 300, 60
    cache, marks = evict_case(gsi, BF, 3, 16, 16, [n], budget, recent=20, sinks=4, offsets=[50], weights=lambda w: -w.abs())
    # (the places are drawn among n + 50 positions: those of the last 20 and first 4 that there are all stay)
    assert (marks.place >= 0).all()


def test_evict_on_another_stream_and_in_a_graph(gsi):
    g = gen(9)
    table, pages = paged([300, 90], 16, 0, g)
    cache = gsi.PagedCache.empty(pages, 2, 16, 64)
    cache.K.normal_(generator=g), cache.V.normal_(generator=g)
    K, V, W = cache.K.clone(), cache.V.clone(), torch.randn(pages, 2, 16, device="cuda", generator=g)
    P = torch.arange(pages * 32, device="cuda").int().view(pages, 2, 16)
    marks = gsi.KeyMarks(W.clone(), P.clone())
    lens, tab = i32([300, 90]), i32(table)
    kept, out = gsi.cache_evict(cache, lens, tab, marks, 64)
    ref = [t.clone() for t in (cache.K, cache.V, marks.weight, marks.place, kept, out)]
    s = torch.cuda.Stream()
    work = gsi.new_workspace(gsi.cache_evict_workspace_size(cache, 2, 64))

    def reset():
        cache.K.copy_(K), cache.V.copy_(V), marks.weight.copy_(W), marks.place.copy_(P), kept.zero_(), out.zero_()

    reset()
    s.wait_stream(torch.cuda.current_stream())
    gsi.cache_evict(cache, lens, tab, marks, 64, kept=kept, offsets_out=out, workspace=work, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (cache.K, cache.V, marks.weight, marks.place, kept, out)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gsi.cache_evict(cache, lens, tab, marks, 64, kept=kept, offsets_out=out, workspace=work)
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, (cache.K, cache.V, marks.weight, marks.place, kept, out)))


def test_offsets_beyond_32_bits(gsi):
    # a cache of more than 2^31 elements, the request's pages at its far end and at its beginning
    hkv, D, page, k, hq = 8, 128, 64, 300, 16
    n_pages = 2**31 // (hkv * D * page) + 40
    big = gsi.PagedCache(*(torch.empty(n_pages, hkv, page, D, dtype=BF, device="cuda") for _ in range(2)))
    table, order = i32([[n_pages - 1, 0, n_pages - 7, n_pages - 2, 3]]), i32([[0, 1, 2, 3, 4]])
    small = gsi.PagedCache(*(torch.randn(5, hkv, page, D, device="cuda", generator=gen(6)).to(BF) for _ in range(2)))
    at = table[0].long()
    big.K[at], big.V[at] = small.K, small.V
    bm, sm = gsi.KeyMarks.empty(big), gsi.KeyMarks.empty(small)
    for q in (1, 130):
        Q = torch.randn(q, hq, D, device="cuda", generator=gen(q)).to(BF)
        lse = torch.empty(q, hq, device="cuda")
        gsi.paged_attention(small, Q, i32([0, q]), i32([k]), order, lse=lse)
        gsi.key_weights(big, Q, lse, i32([0, q]), i32([k]), table, bm)
        gsi.key_weights(small, Q, lse, i32([0, q]), i32([k]), order, sm)
        seen = torch.arange(5 * page, device="cuda").view(5, 1, page).expand(5, hkv, page) < k
        assert torch.equal(bm.weight[at][seen], sm.weight[seen]) and torch.equal(bm.place[at][seen], sm.place[seen])
    for budget in (299, 77):
        kept, _ = gsi.cache_evict(big, i32([k]), table, bm, budget, 10, 2)
        gsi.cache_evict(small, i32([k]), order, sm, budget, 10, 2)
        seen = torch.arange(5 * page, device="cuda").view(5, 1, page).expand(5, hkv, page) < k
        assert kept.item() == budget and torch.equal(big.K[at], small.K) and torch.equal(big.V[at], small.V)
        assert torch.equal(bm.weight[at][seen], sm.weight[seen]) and torch.equal(bm.place[at][seen], sm.place[seen])
        k = budget
    rows = torch.randn(1, (hq + 2 * hkv) * D, device="cuda", generator=gen(1))
    gsi.rotary_append(big, rows, torch.tensor([n_pages * page - 1], device="cuda"), i32([9]), hq, gsi.Rotary.make(D))
    gsi.rotary_append(small, rows, torch.tensor([7], device="cuda"), i32([9]), hq, gsi.Rotary.make(D))
    assert torch.equal(big.K[-1, :, -1], small.K[0, :, 7]) and torch.equal(big.V[-1, :, -1], small.V[0, :, 7])


def test_wide_probability_rows_beyond_32_bits(gsi):
    # rows more than 2^31 elements into the probabilities
    N, V = 4, 3000
    stride = 2**30
    wide = torch.empty((N - 1) * stride + V, dtype=BF, device="cuda")
    target = wide.as_strided((N, V), (stride, 1))
    p = torch.softmax(3 * torch.randn(N, V, device="cuda", generator=gen(2)), -1).to(BF)
    target.copy_(p)
    tokens, u, v = i32([0, 5, int(p[1].argmax()), 7]), torch.tensor([0.0, 0.0, 0.999, 0.5], device="cuda"), torch.tensor([0.3], device="cuda")
    tokens[1] = p[0].argmax().int()
    a, b = (gsi.verify_drafts(t, None, tokens, u, v, i32([0, 4])) for t in (target, p))
    assert torch.equal(a.out, b.out) and a.accepted.tolist() == b.accepted.tolist() == [2]


# ------------------------------------------------------------------ drafts
def verify_case(gsi, n, V, tdt=F, ddt=F, seed=0, near=1.0, edit=None, stride=0, kv=True):
    g = gen(seed)
    N = sum(m + 1 for m in n if m >= 0)
    logits = 3 * torch.randn(N, V, device="cuda", generator=g)
    wide = lambda p, dt: torch.cat([p, torch.full((N, stride), 9.0, device="cuda")], 1).to(dt)[:, :V]  # noqa: E731
    target = wide(torch.softmax(logits, -1), tdt)
    draft = None if ddt is None else wide(torch.softmax(logits + near * torch.randn(N, V, device="cuda", generator=g), -1), ddt)
    tokens = torch.randint(0, V, (N,), device="cuda", generator=g).int()
    if N > 1:
        src = target if draft is None else draft
        tokens[1:] = torch.multinomial(src[:-1].float(), 1, generator=g)[:, 0].int()
    u, v = torch.rand(N, device="cuda", generator=g), torch.rand(len(n), device="cuda", generator=g)
    q_start = np.concatenate([[0], np.cumsum([m + 1 for m in n])])
    kv_len = [100 + r for r in range(len(n))]
    if edit:
        edit(target, draft, tokens, u, v)
    out = torch.full((N,), -9, dtype=torch.int32, device="cuda")
    got = gsi.verify_drafts(target, draft, tokens, u, v, i32(q_start), kv_len=i32(kv_len) if kv else None, out=out)
    want = co.verify(f64(target), None if draft is None else f64(draft), tokens.tolist(), u.tolist(), v.tolist(), q_start, kv_len if kv else None)
    assert got.out.tolist() == [-9 if w is None else w for w in want[0]]
    assert got.accepted.tolist() == want[1]
    assert (got.kept is None and not kv) or got.kept.tolist() == want[2]
    return got


@pytest.mark.parametrize("tdt,ddt", [(F, F), (BF, BF), (F, BF), (BF, F), (F, None), (BF, None)])
@pytest.mark.parametrize("n,V", [([0], 1), ([1], 2), ([3, 0, 1], 7), ([4, 4], 1000), ([7, -1, 2, 0], 4097), ([3], 50257), ([5] * 40, 300)])
def test_verify(gsi, tdt, ddt, n, V):
    verify_case(gsi, n, V, tdt, ddt)
    verify_case(gsi, n, V, tdt, ddt, seed=5, near=0.2, stride=3, kv=False)


def test_verify_many_drafts_and_blocks(gsi):
    assert verify_case(gsi, [700, 3, 600], 64, near=0.0).accepted.tolist() == [700, 3, 600]  # equal probabilities: all stand
    verify_case(gsi, [2] * 200, 9000, seed=2)
    verify_case(gsi, [2], 300_001, seed=3)


def test_verify_leaves_rows_of_no_request(gsi):
    target = torch.softmax(torch.randn(9, 50, device="cuda", generator=gen(8)), -1)
    tokens, u, v = i32(range(9)), torch.full((9,), 2.0, device="cuda"), torch.tensor([0.5, 0.5], device="cuda")
    out = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    got = gsi.verify_drafts(target, None, tokens, u, v, i32([2, 4, 7]), out=out)
    assert got.accepted.tolist() == [0, 0] and out[[0, 1, 7, 8]].tolist() == [-7] * 4 and out[[3, 5, 6]].tolist() == [-1] * 3
    none = gsi.verify_drafts(target[:0], None, tokens[:0], u[:0], v, i32([0, 0, 0]), kv_len=i32([5, 6]))
    assert none.accepted.tolist() == [0, 0] and none.kept.tolist() == [5, 6]


def test_verify_borders(gsi):
    t = torch.tensor([[0.25, 0.25, 0.0, 0.5]], device="cuda")
    for v, want in [(0.0, 0), (0.2499999, 0), (0.25, 1), (0.4999, 1), (0.5, 3), (0.99999994, 3), (1.0, 3), (7.0, 3), (-1.0, 0), (float("nan"), 0)]:
        got = gsi.verify_drafts(t, None, i32([0]), torch.zeros(1, device="cuda"), torch.tensor([v], device="cuda"), i32([0, 1]))
        assert got.out.tolist() == [want], v
    # u q < p strictly: a tie does not stand
    p, q = torch.tensor([[0.25, 0.75], [1.0, 0.0]], device="cuda"), torch.tensor([[0.5, 0.5], [0.0, 0.0]], device="cuda")
    for u, n in [(0.5, 0), (0.49999997, 1), (0.0, 1), (float("nan"), 0)]:
        got = gsi.verify_drafts(p, q, i32([0, 0]), torch.tensor([u, 0.0], device="cuda"), torch.tensor([0.5], device="cuda"), i32([0, 2]))
        assert got.accepted.tolist() == [n] and got.out.tolist() == ([0, 0] if n else [1, -1])


def test_verify_odd_rows(gsi):
    def bad_tokens(target, draft, tokens, u, v):
        tokens[1], tokens[3] = -1, 10**6

    def odd(target, draft, tokens, u, v):
        target[0, 1], target[1, 0], target[2, 3] = float("nan"), -0.5, float("inf")
        if draft is not None:
            draft[0, 2], draft[1, 4] = float("nan"), -1.0

    def same(target, draft, tokens, u, v):  # a rejected draft that leaves nothing: the target itself
        draft[:] = target
        u[:] = 1.0

    def empty(target, draft, tokens, u, v):
        target[:] = 0.0
    for ddt in (F, None):
        verify_case(gsi, [1, 1, 0], 9, ddt=ddt, edit=bad_tokens)
        verify_case(gsi, [1, 1, 0], 9, ddt=ddt, edit=odd)
        assert verify_case(gsi, [1, 1, 0], 9, ddt=ddt, edit=empty).out.tolist() == [-1] * 5
    verify_case(gsi, [1, 2, 0], 9000, edit=same)


def test_verify_follows_the_distribution(gsi):
    # accepted or replaced, the first token comes out as the target has it
    R, V = 60_000, 8
    g = gen(1)
    p, q = torch.softmax(torch.randn(2, V, device="cuda", generator=g), -1)
    tokens = torch.stack([torch.zeros(R, device="cuda").long(), torch.multinomial(q.expand(R, V), 1, generator=g)[:, 0]], 1).flatten().int()
    rows = p.repeat(2 * R, 1)
    got = gsi.verify_drafts(rows, q.repeat(2 * R, 1), tokens, torch.rand(2 * R, device="cuda", generator=g),
                            torch.rand(R, device="cuda", generator=g), torch.arange(R + 1, device="cuda").int() * 2)
    share = torch.bincount(got.out.view(R, 2)[:, 0].long(), minlength=V) / R
    assert ((share - p).abs() <= 6 * (p * (1 - p) / R).sqrt()).all()  # six standard deviations


# ------------------------------------------------------------------ pages given back
def trim_case(gsi, kv_len, kept, page, width, n_free, capacity, seed=0):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(len(kv_len) * width + capacity).astype(np.int32)
    table, free = ids[:len(kv_len) * width].reshape(len(kv_len), width), ids[len(kv_len) * width:]
    f = i32(free)
    left, status = gsi.paged_trim(i32(kv_len), i32(kept), i32(table).view(len(kv_len), width), f, i32([n_free]), page)
    want = co.trim(kv_len, kept, table, free, n_free, page)
    assert f.tolist() == want[0] and left.item() == want[1] and status.item() == want[2]
    return want


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("R,most,back", [(1, 1, 1), (1, 5000, 5000), (7, 40, 3), (513, 300, 300), (4099, 60, 60), (9000, 40, 20)])
def test_trim(gsi, page, R, most, back):
    rng = np.random.default_rng(R + page)
    kv = rng.integers(0, most + 1, R)
    kept = np.maximum(0, kv - rng.integers(0, back + 1, R))
    n = int((-(-kv // page) - -(-kept // page)).sum())
    assert trim_case(gsi, kv.tolist(), kept.tolist(), page, max(1, -(-most // page)), 3, n + 3)[2] == 0
    assert trim_case(gsi, kv.tolist(), kept.tolist(), page, max(1, -(-most // page)), 0, n + 40)[2] == 0
    if n:
        assert trim_case(gsi, kv.tolist(), kept.tolist(), page, max(1, -(-most // page)), 4, n + 3)[2] == gsi.PLAN_NO_PAGES


def test_trim_refuses_what_cannot_be(gsi):
    assert trim_case(gsi, [20, 5], [21, 5], 16, 3, 0, 9)[2] == gsi.PLAN_BAD_LENGTH
    assert trim_case(gsi, [20, -5], [2, -5], 16, 3, 0, 9)[2] == gsi.PLAN_BAD_LENGTH
    assert trim_case(gsi, [20, 49], [2, 0], 16, 3, 0, 9)[2] == gsi.PLAN_TABLE_FULL
    assert trim_case(gsi, [20, 5], [2, 0], 16, 3, -1, 9)[2] == gsi.PLAN_NO_PAGES
    assert trim_case(gsi, [20, 5], [2, 0], 16, 3, 10, 9)[2] == gsi.PLAN_NO_PAGES
    assert trim_case(gsi, [49, -1], [2, -1], 16, 3, 10, 9)[2] == 7
    assert trim_case(gsi, [], [], 16, 3, 2, 9)[2] == 0 and trim_case(gsi, [0], [0], 16, 1, 0, 0)[2] == 0


def test_trim_then_plan_takes_the_same_pages(gsi):
    kv = i32([100, 37])
    table = i32([[5, 1, 7, 3, 9, 11, 2], [4, 8, 6, -1, -1, -1, -1]])
    free, n = i32([20, 21] + [-1] * 8), i32([2])
    kept = i32([40, 5])
    n2, status = gsi.paged_trim(kv, kept, table, free, n, 16)
    assert status.item() == 0 and n2.item() == 8
    t2 = table.clone()
    plan = gsi.paged_plan(kept, kv - kept, t2, free, n2, 16, 92)
    assert plan.status.item() == 0 and torch.equal(t2, table) and plan.n_free.item() == 2


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dt,D,turned,layout", [(BF, 128, 128, "half"), (BF, 64, 16, "pairs"), (F, 32, 32, "half")])
def test_steps_of_a_server_with_a_bounded_cache(gsi, dt, D, turned, layout):
    """Prompts and then single tokens: plan, rotary append, attention, weights,
    eviction, return of pages, each against its definition on what it got."""
    hq, hkv, page, budget, R = 4, 2, 16, 48, 3
    g = gen(D)
    pages = 24
    cache = gsi.PagedCache(*(torch.zeros(pages, hkv, page, D, dtype=dt, device="cuda") for _ in range(2)))
    marks = gsi.KeyMarks(torch.zeros(pages, hkv, page, device="cuda"), torch.zeros(pages, hkv, page, dtype=torch.int32, device="cuda"))
    turn = gsi.Rotary.make(turned, layout=layout, scaling="linear", factor=4.0)
    table, free, n_free = torch.full((R, 8), -1, dtype=torch.int32, device="cuda"), i32(range(pages)), i32([pages])
    cached, gone = i32([0] * R), i32([0] * R)
    work = gsi.new_workspace(max(gsi.paged_attention_workspace_size(cache, hq), gsi.key_weights_workspace_size(),
                                 gsi.cache_evict_workspace_size(cache, R, budget)))
    lengths = np.zeros(R, dtype=int)
    for step, fresh in enumerate([[70, 30, 5], [1, 1, 1], [1, 0, 60], [2, 40, 1], [1, 1, 1]]):
        T = sum(fresh)
        lengths += fresh
        plan = gsi.paged_plan(cached, i32(fresh), table, free, n_free, page, T)
        rows = torch.randn(T, (hq + 2 * hkv) * D, device="cuda", generator=g)
        q = gsi.rotary_append(cache, rows, plan.slots, plan.positions, hq, turn, token_req=plan.token_req, offsets=gone)
        # the positions are those of the sequences, whatever has left the cache
        want_pos = np.concatenate([np.arange(n - f, n) for n, f in zip(lengths, fresh)])
        ref = co.rotary(f64(rows).reshape(T, -1, D)[:, :hq], want_pos, co.Angle(turn.phases.tolist()), layout, turn.scale)
        assert np.abs(f64(q) - ref).max() <= 2**-18 + (2**-8 * np.abs(ref).max() if dt is BF else 0)
        lse = torch.empty(T, hq, device="cuda")
        gsi.paged_attention(cache, q, plan.q_start, plan.kv_len, table, max_q=max(fresh), workspace=work, lse=lse)
        before = f64(marks.weight), marks.place.cpu().numpy()
        gsi.key_weights(cache, q, lse, plan.q_start, plan.kv_len, table, marks, held=cached, offsets=gone, max_q=max(fresh), workspace=work)
        w, p = co.key_weights(f64(q), f64(cache.K), f64(lse), plan.q_start.tolist(), plan.kv_len.tolist(), cached.tolist(), gone.tolist(),
                              table.cpu().numpy(), *before, D**-0.5)
        assert np.array_equal(p, marks.place.cpu().numpy()) and np.allclose(f64(marks.weight), w, rtol=1e-4, atol=0)
        before = [f64(cache.K), f64(cache.V), f64(marks.weight), marks.place.cpu().numpy()]
        kept, out = gsi.cache_evict(cache, plan.kv_len, table, marks, budget, recent=8, sinks=2, offsets=gone, workspace=work)
        want = co.evict(before[0], before[1], plan.kv_len.tolist(), table.cpu().numpy(), before[2], before[3], budget, 8, 2, gone.tolist())
        for a, b in zip((f64(cache.K), f64(cache.V), f64(marks.weight), marks.place.cpu().numpy(), kept.tolist(), out.tolist()), want):
            assert np.array_equal(np.asarray(a), np.asarray(b))
        n_free, status = gsi.paged_trim(plan.kv_len, kept, table, free, plan.n_free, page)
        assert plan.status.item() == 0 and status.item() == 0
        cached, gone = kept, out
        assert (f64(cached) + f64(gone) == lengths).all()
        held = [-(-int(n) // page) for n in cached.tolist()]
        mine = [int(table[r, j]) for r in range(R) for j in range(held[r])] + free[:int(n_free)].tolist()
        assert sorted(mine) == list(range(pages))  # no page lost, none twice
        for r in range(R):  # the places held are different positions of the sequence, the last eight and first two among them
            for h in range(hkv):
                at = [int(marks.place[int(table[r, j // page]), h, j % page]) for j in range(int(cached[r]))]
                assert len(set(at)) == len(at)
                if lengths[r] > budget:
                    assert set(range(lengths[r] - 8, lengths[r])) | {0, 1} <= set(at)


def test_drafted_steps_in_one_graph(gsi):
    """Verification and the return of pages, captured and replayed with other numbers."""
    g = gen(4)
    R, n, V, page = 5, 3, 1000, 16
    N = R * (n + 1)
    target = torch.softmax(3 * torch.randn(N, V, device="cuda", generator=g), -1)
    draft = torch.softmax(3 * torch.randn(N, V, device="cuda", generator=g), -1)
    tokens, u, v = torch.randint(0, V, (N,), device="cuda", generator=g).int(), torch.rand(N, device="cuda"), torch.rand(R, device="cuda")
    q_start, kv = torch.arange(R + 1, device="cuda").int() * (n + 1), i32([33, 49, 20, 17, 64])
    table, free, n_free = torch.arange(R * 4, device="cuda").int().view(R, 4), i32([-1] * 20), i32([0])
    out, acc, kept, left, status = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (N, R, R, 1, 1))

    def step():
        gsi.verify_drafts(target, draft, tokens, u, v, q_start, kv_len=kv, out=out, accepted=acc, kept=kept)
        gsi.paged_trim(kv, kept, table, free, n_free, page, n_free_out=left, status=status)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        h = gen(seed)
        u.uniform_(generator=h), v.uniform_(generator=h)
        free.fill_(-1)
        if seed % 2:
            target.copy_(draft)
        graph.replay()
        torch.cuda.synchronize()
        want = co.verify(f64(target), f64(draft), tokens.tolist(), u.tolist(), v.tolist(), q_start.tolist(), kv.tolist())
        assert out.tolist() == want[0] and acc.tolist() == want[1] and kept.tolist() == want[2]
        w = co.trim(kv.tolist(), want[2], table.cpu().numpy(), [-1] * 20, 0, page)
        assert free.tolist() == w[0] and left.item() == w[1] and status.item() == 0


def test_rotary_verify_and_trim_on_another_stream(gsi):
    s = torch.cuda.Stream()
    rows, slots, pos = torch.randn(9, 6 * 64, device="cuda", generator=gen(3)), torch.randperm(32, device="cuda", generator=gen(4))[:9], i32(range(50, 59))
    a, b = (gsi.PagedCache(*(torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda") for _ in range(2))) for _ in range(2))
    turn = gsi.Rotary.make(64)
    target, tokens = torch.softmax(torch.randn(6, 500, device="cuda", generator=gen(5)), -1), i32([0, 3, 9, 1, 4, 400])
    u, v, qs, kv = torch.rand(6, device="cuda"), torch.rand(2, device="cuda"), i32([0, 4, 6]), i32([40, 60])
    table, free = i32([[1, 2, 3, 9], [4, 5, 6, 8]]), [i32([-1] * 8) for _ in range(2)]
    torch.cuda.synchronize()
    q = gsi.rotary_append(a, rows, slots, pos, 2, turn)
    r = gsi.verify_drafts(target, None, tokens, u, v, qs, kv_len=kv)
    n = gsi.paged_trim(kv, i32([3, 0]), table, free[0], i32([0]), 16)
    kept = i32([3, 0])
    zero = i32([0])
    torch.cuda.synchronize()
    q2 = gsi.rotary_append(b, rows, slots, pos, 2, turn, stream=s)
    r2 = gsi.verify_drafts(target, None, tokens, u, v, qs, kv_len=kv, stream=s)
    n2 = gsi.paged_trim(kv, kept, table, free[1], zero, 16, stream=s)
    s.synchronize()
    assert torch.equal(q, q2) and torch.equal(a.K, b.K) and torch.equal(a.V, b.V)
    assert torch.equal(r.out, r2.out) and torch.equal(r.accepted, r2.accepted) and torch.equal(r.kept, r2.kept)
    assert torch.equal(free[0], free[1]) and n[0].item() == n2[0].item() == 6


def test_tensors_elsewhere_are_refused(gsi):
    cache = gsi.PagedCache.empty(4, 2, 16, 64)
    marks = gsi.KeyMarks.empty(cache)
    with pytest.raises(ValueError):
        gsi.cache_evict(cache, torch.zeros(1, dtype=torch.int32), i32([[0]]), marks, 4)
    with pytest.raises(ValueError):
        gsi.cache_evict(cache, i32([0]), i32([[0]]), gsi.KeyMarks(marks.weight[:2], marks.place[:2]), 4)
    with pytest.raises(ValueError):
        gsi.verify_drafts(torch.zeros(2, 4), None, i32([0, 0]), torch.zeros(2, device="cuda"), torch.zeros(1, device="cuda"), i32([0, 2]))
    with pytest.raises(ValueError):
        gsi.paged_trim(i32([1]), torch.zeros(1, dtype=torch.int32), i32([[0]]), i32([0]), i32([0]), 16)
    with pytest.raises(ValueError):
        gsi.rotary_append(cache, torch.zeros(1, 6 * 64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"),
                          torch.zeros(1, dtype=torch.int32), 2, gsi.Rotary.make(64))
    with pytest.raises(gsi.GsiError):
        gsi.cache_evict(cache, i32([0]), i32([[0]]), marks, 4, recent=3, sinks=2)
