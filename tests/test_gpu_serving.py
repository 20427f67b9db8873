"""Serving operators on the GPU against their float64 definitions.

Tolerances, from the arithmetic the kernels do:
  * plan: whole numbers, equal;
  * append: a copy, or one rounding to nearest even: equal bit for bit;
  * attention: an output is a convex combination of the visible values, so a
    relative error e of the weights moves it by at most e * sum_j p_j |v_j| =
    e A.  float32: scores of magnitude <= ~20 from up to 256 products, rounded
    at 2^-24 each in random directions (sqrt(256) * 2^-24 * 20 = 2e-5), the
    exponential's few ulps and the sum's rounding: e = 1e-4 covers them five
    times.  bf16 maps: weights rounded to bf16, whose 8 significant bits make
    that a relative error of up to 2^-8, and the result rounded once (up to
    2^-8 |o|): 2^-8 A + 2^-8 |o| + 1e-4 A;
  * norm: sums of up to 16384 squares in a tree of short chains (relative
    error under 40 * 2^-24 = 2.4e-6), centred values and products: 2e-5 (1 +
    |value|) for rows of magnitude ~1 whose mean is at most a few standard
    deviations; a bf16 output adds 2^-8 |value|.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so

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


# ------------------------------------------------------------------ plan
def plan_case(gsi, cached, fresh, page, width, n_free, n_tokens, seed=0, capacity=None):
    rng = np.random.default_rng(seed)
    held = [max(0, -(-c // page)) for c in cached]
    ids = rng.permutation(sum(held) + max(n_free, capacity or 0, 1) + 3).astype(np.int32)
    table = np.full((len(cached), width), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(held):
        n = min(n, width)
        table[r, :n] = ids[at:at + n]
        at += n
    free = ids[sum(held):sum(held) + (capacity if capacity is not None else max(n_free, 0))]
    tab = torch.tensor(table, device="cuda")
    got = gsi.paged_plan(i32(cached), i32(fresh), tab, i32(free), i32([n_free]), page, n_tokens)
    want = so.paged_plan(cached, fresh, table, free, n_free, page, n_tokens)
    for g, w, name in zip((got.q_start, got.kv_len, got.slots, got.token_req, got.positions, tab, got.n_free,
                           got.status), want, ("q_start", "kv_len", "slots", "token_req", "positions", "table",
                                               "n_free", "status")):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w, dtype=np.int64).reshape(-1)), name
    return want


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("R,most_cached,most_fresh", [(1, 0, 1), (1, 700, 300), (7, 40, 3), (33, 500, 90),
                                                      (513, 300, 40), (4099, 60, 5), (9000, 40, 3)])
def test_plan(gsi, page, R, most_cached, most_fresh):
    rng = np.random.default_rng(R + page)
    cached, fresh = rng.integers(0, most_cached + 1, R).tolist(), rng.integers(0, most_fresh + 1, R).tolist()
    want = sum(-(-(c + f) // page) - -(-c // page) for c, f in zip(cached, fresh))
    width = max(-(-(c + f) // page) for c, f in zip(cached, fresh)) + 1
    plan_case(gsi, cached, fresh, page, width, want + 2, sum(fresh) + 5)
    assert plan_case(gsi, cached, fresh, page, width, want, sum(fresh))[7] == 0


def test_plan_refuses_what_does_not_fit(gsi):
    assert plan_case(gsi, [0, 5], [17, 20], 16, 4, 2, 40)[7] == gsi.PLAN_NO_PAGES
    assert plan_case(gsi, [0, 5], [17, 20], 16, 1, 4, 40)[7] == gsi.PLAN_TABLE_FULL
    assert plan_case(gsi, [0, -5], [17, 20], 16, 4, 4, 40)[7] == gsi.PLAN_BAD_LENGTH
    assert plan_case(gsi, [0, 5], [17, -1], 16, 4, 4, 40)[7] == gsi.PLAN_BAD_LENGTH
    assert plan_case(gsi, [0, 2**31 - 5], [17, 9], 16, 4, 4, 40)[7] == gsi.PLAN_BAD_LENGTH
    assert plan_case(gsi, [0, 5], [17, 20], 16, 4, 4, 36)[7] == gsi.PLAN_TOO_MANY_TOKENS
    assert plan_case(gsi, [0, 5], [17, 20], 16, 4, -1, 40, capacity=4)[7] == gsi.PLAN_NO_PAGES
    assert plan_case(gsi, [0, 5], [17, 20], 16, 4, 9, 40, capacity=4)[7] == gsi.PLAN_NO_PAGES
    assert plan_case(gsi, [0, 5], [30, 30], 16, 1, 0, 9)[7] == 2 | 4 | 8


def test_plan_without_requests_or_tokens(gsi):
    assert plan_case(gsi, [], [], 16, 2, 3, 4)[7] == 0
    assert plan_case(gsi, [], [], 16, 2, 3, 0)[7] == 0
    assert plan_case(gsi, [3, 0], [0, 0], 16, 2, 3, 0)[7] == 0


def test_plan_of_a_caller_without_a_page(gsi):
    # a table that says -1 for a page a request should hold: the tokens of that page have no slot
    tab = i32([[-1, -1]])
    p = gsi.paged_plan(i32([5]), i32([13]), tab, i32([9]), i32([1]), 16, 13)
    assert p.status.item() == 0 and p.slots.tolist() == [-1] * 11 + [144, 145] and tab.tolist() == [[-1, 9]]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("xdt,cdt", [(F, BF), (BF, BF), (F, F), (BF, F)])
@pytest.mark.parametrize("T,hq,hkv,D,page", [(1, 2, 1, 64, 16), (5, 3, 3, 80, 32), (37, 8, 2, 128, 16),
                                             (300, 4, 4, 256, 256), (3, 0, 2, 16, 64)])
def test_append(gsi, xdt, cdt, T, hq, hkv, D, page):
    g = torch.Generator(device="cuda").manual_seed(T)
    wide = torch.randn(T, (hq + 2 * hkv) * D + 24, device="cuda", generator=g).to(xdt)
    rows = wide[:, 16:16 + (hq + 2 * hkv) * D]  # a view with a stride of its own
    pages = 2 * -(-T // page) + 1
    cache = gsi.PagedCache.empty(pages, hkv, page, D, cdt)
    cache.K.normal_(generator=g), cache.V.normal_(generator=g)
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:T]
    slots[T // 2] = -1 if T % 2 else pages * page  # padding, or out of the cache: the cache stays
    K, V = cache.K.clone(), cache.V.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            K[s // page, :, s % page] = rows[t, hq * D:(hq + hkv) * D].view(hkv, D).to(cdt)
            V[s // page, :, s % page] = rows[t, (hq + hkv) * D:].view(hkv, D).to(cdt)
    Q = gsi.cache_append(cache, rows, slots, hq)
    assert torch.equal(cache.K, K) and torch.equal(cache.V, V)
    assert torch.equal(Q, rows[:, :hq * D].reshape(T, hq, D).to(cdt))


def test_append_into_another_layout(gsi):
    K, V = (torch.zeros(4, 16, 3, 32, dtype=BF, device="cuda") for _ in range(2))
    cache = gsi.PagedCache(K.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3))
    rows = torch.randn(7, 8 * 32, device="cuda")
    slots = torch.arange(7, device="cuda") * 9 + 1
    gsi.cache_append(cache, rows, slots, 2)
    for t in range(7):
        assert torch.equal(K.view(64, 3, 32)[t * 9 + 1], rows[t, 64:160].view(3, 32).to(BF))
        assert torch.equal(V.view(64, 3, 32)[t * 9 + 1], rows[t, 160:].view(3, 32).to(BF))
    assert K.count_nonzero() == 7 * 96


def test_append_of_nothing(gsi):
    cache = gsi.PagedCache.empty(1, 2, 16, 64)
    assert gsi.cache_append(cache, torch.empty(0, 6 * 64, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"),
                            2).shape == (0, 2, 64)


# ------------------------------------------------------------------ attention
def pages_for(lens, page, width, seed, spare=3):
    """A table of scattered pages, -1 where a request has none, and the number of pages."""
    rng = np.random.default_rng(seed)
    n = sum(-(-max(0, k) // page) for _, k in lens) + spare
    ids = rng.permutation(n)
    table, at = np.full((len(lens), width), -1, dtype=np.int32), 0
    for r, (_, k) in enumerate(lens):
        m = min(-(-max(0, k) // page), width)
        table[r, :m] = ids[at:at + m]
        at += m
    return table, n


def attention_case(gsi, dt, hq, hkv, D, page, lens, causal=True, window=0, seed=0, permuted=False, width=None,
                   scale=None, touch=None, max_q=None, pad=(0, 0), workspace=None, qscale=2.0):
    """lens: (new tokens, keys) of each request.  Slots that hold no key of a
    request are NaN in K and V.  touch(Q, K, V, table, key_at): changes inputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = max([-(-k // page) for _, k in lens] + [1]) if width is None else width
    table, n_pages = pages_for(lens, page, width, seed)
    shape = (n_pages, page, hkv, D) if permuted else (n_pages, hkv, page, D)
    K, V = (torch.full(shape, float("nan"), dtype=dt, device="cuda") for _ in range(2))
    if permuted:
        K, V = K.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3)

    def key_at(r, j):
        return int(table[r, j // page]), j % page

    for r, (_, k) in enumerate(lens):
        k = min(k, width * page)
        for j in range(0, k, page):
            pg, n = int(table[r, j // page]), min(page, k - j)
            K[pg, :, :n] = torch.randn(hkv, n, D, device="cuda", generator=g).to(dt)
            V[pg, :, :n] = torch.randn(hkv, n, D, device="cuda", generator=g).to(dt)
    q_start = np.cumsum([pad[0]] + [q for q, _ in lens])
    N = int(q_start[-1]) + pad[1]
    wide = (torch.randn(N, hq * D + 32, device="cuda", generator=g) * qscale).to(dt)
    Q = wide[:, :hq * D].view(N, hq, D) if N else wide[:, :hq * D].reshape(N, hq, D)
    if touch:
        touch(Q, K, V, table, key_at)
    cache = gsi.PagedCache(K, V)
    out = torch.full((N, hq, D), 7.0, dtype=dt, device="cuda")
    gsi.paged_attention(cache, Q, i32(q_start), i32([k for _, k in lens]), torch.tensor(table, device="cuda"),
                        causal=causal, window=window, scale=scale, out=out, max_q=max_q, workspace=workspace)
    O, A, rows = so.attention(f64(Q), f64(K), f64(V), q_start, [k for _, k in lens], table,
                              D ** -0.5 if scale is None else scale, causal, window)
    o = f64(out)
    assert (o[~rows] == 7.0).all(), "rows of no request were written"
    fin = np.isfinite(O[rows])
    assert np.array_equal(o[rows][~fin], O[rows][~fin], equal_nan=True), "NaN or infinities unlike the definition's"
    o, O_, A = o[rows][fin], O[rows][fin], A[rows][fin]
    err, tol = np.abs(o - O_), 1e-4 * A + (0 if dt == F else 2**-8 * (A + np.abs(O_)))
    if err.size:
        assert (err <= tol).all(), f"{float((err / np.maximum(tol, 1e-30)).max())} times the tolerance"
    return out, O


LENS = [
    [(1, 1)], [(1, 17)], [(2, 2)], [(1, 0), (1, 300)],                     # one token, no key at all
    [(1, 5), (1, 64), (1, 129), (1, 1000)],                                # decode, ragged
    [(16, 16), (3, 40)], [(5, 131), (1, 700), (0, 50), (33, 33)],          # chunks and a request without new tokens
    [(200, 200)], [(130, 515), (7, 1290)], [(4, 2), (6, 0)],               # tiles, more tokens than keys (empty rows)
]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dt,hq,hkv,D,page", [(BF, 2, 2, 128, 16), (BF, 8, 2, 64, 32), (BF, 2, 2, 256, 64),
                                              (BF, 6, 2, 80, 16), (BF, 5, 1, 128, 128), (BF, 3, 1, 192, 256),
                                              (F, 2, 2, 64, 16), (F, 6, 2, 32, 32), (F, 2, 1, 256, 64)])
def test_attention(gsi, lens, dt, hq, hkv, D, page):
    attention_case(gsi, dt, hq, hkv, D, page, lens)


@pytest.mark.parametrize("dt,D", [(BF, 8), (BF, 16), (BF, 40), (BF, 136), (F, 4), (F, 8), (F, 20), (F, 100), (F, 252)])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 3)], [(3, 200), (1, 1)], [(70, 300)]], ids=str)
def test_attention_odd_head_sizes(gsi, dt, D, lens):
    attention_case(gsi, dt, 4, 2, D, 16, lens)


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 256), (F, 64)])
@pytest.mark.parametrize("window", [1, 16, 100, 128, 1000])
@pytest.mark.parametrize("lens", [[(1, 1), (1, 500), (2, 131)], [(150, 400), (3, 129)]], ids=str)
def test_attention_window(gsi, dt, D, window, lens):
    attention_case(gsi, dt, 4, 2, D, 16, lens, window=window)


@pytest.mark.parametrize("dt,D", [(BF, 64), (BF, 256), (F, 128)])
@pytest.mark.parametrize("lens", [[(1, 77), (1, 0)], [(40, 9), (150, 300), (3, 0)], [(9, 1000)]], ids=str)
def test_attention_not_causal(gsi, dt, D, lens):
    attention_case(gsi, dt, 4, 2, D, 32, lens, causal=False)


@pytest.mark.parametrize("dt", [BF, F])
def test_attention_layout_padding_and_scale(gsi, dt):
    lens = [(3, 100), (40, 170)]
    attention_case(gsi, dt, 4, 2, 64, 32, lens, permuted=True, pad=(2, 5), scale=0.3)
    attention_case(gsi, dt, 4, 2, 64, 32, lens, scale=-0.1)
    attention_case(gsi, dt, 4, 2, 64, 32, lens, scale=0.0)
    attention_case(gsi, dt, 4, 2, 64, 32, lens, max_q=1)  # a wrong hint costs time, not results
    attention_case(gsi, dt, 4, 2, 64, 32, [(1, 100)] * 3, max_q=1000)
    attention_case(gsi, dt, 128, 1, 64, 16, [(2, 40)])    # as many heads a key/value head as there can be
    attention_case(gsi, dt, 50, 1, 64, 16, [(9, 200)])


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 256), (F, 64)])
@pytest.mark.parametrize("lens", [[(1, 3000)], [(1, 9000), (1, 10)], [(20, 5000)]], ids=str)
def test_attention_long(gsi, dt, D, lens):
    attention_case(gsi, dt, 2, 1, D, 64, lens)


@pytest.mark.parametrize("dt,hq,hkv,D,page,lens,window", [
    (BF, 16, 16, 128, 16, [(700, 3000), (60, 2000)], 0), (BF, 16, 8, 64, 64, [(600, 600), (513, 2000)], 0),
    (BF, 12, 12, 256, 32, [(400, 2300), (130, 131)], 0), (BF, 8, 8, 192, 128, [(500, 1500)], 0),
    (BF, 16, 16, 128, 16, [(900, 1900)], 300), (BF, 8, 8, 256, 64, [(700, 1900)], 200), (BF, 24, 8, 80, 32, [(300, 4000)], 0),
    (BF, 16, 16, 128, 16, [(1, 9000), (1, 3001)], 0), (BF, 16, 2, 256, 64, [(1, 9000), (2, 8000)] * 3, 0),
    (BF, 8, 8, 64, 32, [(1, 20000), (0, 9), (1, 1)], 0), (F, 8, 8, 64, 16, [(150, 1500), (1, 4000)], 0)])
def test_attention_many_tiles_a_cta(gsi, dt, hq, hkv, D, page, lens, window):
    attention_case(gsi, dt, hq, hkv, D, page, lens, window=window)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("lens", [[(1, 40), (1, 200)], [(140, 300)], [(6, 9)]], ids=str)
def test_attention_table_entries_outside_the_cache(gsi, dt, lens):
    def touch(Q, K, V, table, key_at):
        table[0, 1 if table.shape[1] > 1 and lens[0][1] > 16 else 0] = -1
        table[-1, 0] = K.shape[0] + 5
    attention_case(gsi, dt, 4, 2, 64, 16, lens, touch=touch)


@pytest.mark.parametrize("dt", [BF, F])
def test_attention_keys_beyond_the_table_are_cut(gsi, dt):
    attention_case(gsi, dt, 2, 2, 64, 16, [(1, 100), (4, 70)], width=3)


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 256), (BF, 80), (F, 64)])
@pytest.mark.parametrize("lens,bad", [([(9, 40)], 36), ([(150, 300)], 200), ([(150, 300)], 299), ([(260, 260)], 130),
                                      ([(1, 500), (3, 20)], 18)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["K", "V"])
def test_attention_nonfinite_token_reaches_only_who_sees_it(gsi, dt, D, lens, bad, value, where):
    def touch(Q, K, V, table, key_at):
        pg, o = key_at(len(lens) - 1, bad)
        if where == "V":
            V[pg, :, o, 3:5] = value
        else:
            K[pg, :, o, 3:5] = float("nan")
    out, O = attention_case(gsi, dt, 4, 2, D, 16, lens, touch=touch)
    # the tokens before it, in the same chunk, are finite
    q, k = lens[-1]
    before = bad - (k - q)
    if before > 0:
        first = sum(n for n, _ in lens[:-1])
        assert torch.isfinite(out[first:first + before].float()).all()


@pytest.mark.parametrize("dt,hq,D", [(BF, 4, 64), (BF, 4, 128), (BF, 4, 256), (F, 4, 64), (F, 130, 32)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,bad", [([(9, 40)], 36), ([(150, 300)], 200), ([(1, 500), (3, 20)], 18), ([(40, 40)], 0)], ids=str)
def test_attention_infinite_key(gsi, dt, hq, D, lens, bad, value):
    # scores of both infinities: a row is NaN where the largest one is, and loses the key where it is the smallest
    def touch(Q, K, V, table, key_at):
        pg, o = key_at(len(lens) - 1, bad)
        K[pg, :, o, 3] = value
    attention_case(gsi, dt, hq, 2, D, 16, lens, touch=touch)


@pytest.mark.parametrize("dt,hq,D", [(BF, 4, 64), (BF, 4, 128), (BF, 4, 256), (F, 4, 64), (F, 130, 32)])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 3000), (2, 50)], [(70, 70), (3, 0)], [(300, 900)]], ids=str)
def test_attention_scores_all_lowest(gsi, dt, hq, D, lens, window):
    # every score of every second head is -inf, which is no softmax; a row without a key is zeros all the same
    def touch(Q, K, V, table, key_at):
        K[..., 3] = float("inf")
        Q[:, :, 3] = 1.0
        Q[:, 1::2, 3] = -1.0
    attention_case(gsi, dt, hq, 2, D, 16, lens, window=window, touch=touch)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("lens,window", [([(1, 16)], 0), ([(1, 160), (2, 40)], 0), ([(1, 5000), (1, 7)], 0), ([(150, 150)], 0),
                                         ([(300, 2000), (20, 50)], 0), ([(200, 700)], 100)], ids=str)
@pytest.mark.parametrize("weight", [0.5 * (1 + 0.98 * 2**-8), 0.5 * (1 + 1.02 * 2**-8), 1 + 0.98 * 2**-8, 1 + 1.02 * 2**-8])
def test_attention_of_equal_values_is_the_value(gsi, D, lens, window, weight):
    # A weighted mean of one value is the value.  Most keys have a weight half way between two bf16 values, so all of them
    # are rounded one way for the product over a bf16 cache: the rounded weights have to be the ones that are summed.
    # What is left is the float32 rounding of both sums (under 1e-4), far below that of the result.
    def touch(Q, K, V, table, key_at):
        V[:] = torch.linspace(1.0, 2.0 - 2**-7, D, device="cuda").to(BF)
        Q[:], K[:] = 0, 0
        Q[:, :, 0] = 1.0
        for r, (_, k) in enumerate(lens):
            for j in range(0, k, 16):
                K[key_at(r, j)[0], :, :, 0] = 1.0 if weight < 1 or j >= 128 else 0.0
                K[key_at(r, j)[0], :, 5, 0] = 0.0 if weight < 1 or j < 128 else 1.0
    out, O = attention_case(gsi, BF, 4, 2, D, 16, lens, window=window, touch=touch, scale=float(np.log(weight)))
    assert np.array_equal(f64(out), f64(torch.tensor(O).to(BF)))


@pytest.mark.parametrize("dt", [BF, F])
def test_attention_extreme_scores(gsi, dt):
    # scores of +-1e4: the running maximum grows from tile to tile; scores that fall; all equal
    def rising(Q, K, V, table, key_at):
        Q[:] = 1.0
        for j in range(700):
            pg, o = key_at(0, j)
            K[pg, :, o] = (j - 350) * 0.125
    attention_case(gsi, dt, 2, 2, 64, 16, [(3, 700)], touch=rising)

    def falling(Q, K, V, table, key_at):
        Q[:] = 1.0
        for j in range(700):
            pg, o = key_at(0, j)
            K[pg, :, o] = (350 - j) * 0.125
    attention_case(gsi, dt, 2, 2, 64, 16, [(140, 700)], touch=falling)

    def lowest(Q, K, V, table, key_at):
        Q[:] = 1.0
        K.nan_to_num_(nan=0.0).fill_(-torch.finfo(torch.bfloat16).max / 256)
    attention_case(gsi, dt, 2, 2, 64, 16, [(140, 300), (1, 77)], touch=lowest)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("q,group", [(1, 1), (1, 16), (40, 4)])
def test_attention_streams_from_memory(gsi, D, q, group):
    # more keys than the caches hold: copies land out of order, rings wrap thousands of times
    hkv, page, k = 8, 16, 60001
    n = -(-k // page)
    g = torch.Generator(device="cuda").manual_seed(D + q)
    K, V = (torch.randn(n, hkv, page, D, device="cuda", generator=g, dtype=BF) for _ in range(2))
    Q = 2 * torch.randn(q, hkv * group, D, device="cuda", generator=g, dtype=BF)
    table = torch.randperm(n, device="cuda", generator=g).int()[None]
    ws = gsi.new_workspace(gsi.paged_attention_workspace_size(gsi.PagedCache(K, V), hkv * group))
    out = gsi.paged_attention(gsi.PagedCache(K, V), Q, i32([0, q]), i32([k]), table, workspace=ws)
    assert gsi.workspace_status(ws) == 0
    hidden = torch.arange(k, device="cuda") > torch.arange(k - q, k, device="cuda")[:, None]
    for h in range(hkv * group):
        ks, vs = (t[table[0].long(), h // group].reshape(-1, D)[:k].double() for t in (K, V))
        p = torch.softmax((Q[:, h].double() @ ks.T * D ** -0.5).masked_fill(hidden, -float("inf")), -1)
        want, A = p @ vs, p @ vs.abs()
        assert ((out[:, h].double() - want).abs() <= 1e-4 * A + 2**-8 * (A + want.abs())).all()


@pytest.mark.parametrize("D,hq,hkv,q,k", [(256, 16, 16, 2048, 2048), (128, 32, 32, 1500, 1700), (64, 40, 8, 1900, 1900),
                                           (192, 24, 24, 1601, 1601), (128, 48, 16, 1111, 1300)])
def test_attention_of_one_prompt(gsi, D, hq, hkv, q, k):
    # enough units of one causal request to be dealt out whole
    page = 32
    n = -(-k // page)
    g = torch.Generator(device="cuda").manual_seed(D + q)
    K, V = (torch.randn(n, hkv, page, D, device="cuda", generator=g, dtype=BF) for _ in range(2))
    Q = 2 * torch.randn(q, hq, D, device="cuda", generator=g, dtype=BF)
    table = torch.randperm(n, device="cuda", generator=g).int()[None]
    ws = gsi.new_workspace(gsi.paged_attention_workspace_size(gsi.PagedCache(K, V), hq))
    out = gsi.paged_attention(gsi.PagedCache(K, V), Q, i32([0, q]), i32([k]), table, workspace=ws)
    assert gsi.workspace_status(ws) == 0
    hidden = torch.arange(k, device="cuda") > torch.arange(k - q, k, device="cuda")[:, None]
    for h in range(0, hq, 5):
        ks, vs = (t[table[0].long(), h * hkv // hq].reshape(-1, D)[:k].double() for t in (K, V))
        p = torch.softmax((Q[:, h].double() @ ks.T * D ** -0.5).masked_fill(hidden, -float("inf")), -1)
        want, A = p @ vs, p @ vs.abs()
        assert ((out[:, h].double() - want).abs() <= 1e-4 * A + 2**-8 * (A + want.abs())).all()


@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_attention_units_end_in_step(gsi, D):
    # many short units a CTA, whose last product may end before or after the rows' threads ask for it: no wait gives up,
    # and every run gives the same
    hq, hkv, page, lens = 64, 8, 32, [287, 191, 95, 250, 154, 58, 213]
    g = torch.Generator(device="cuda").manual_seed(D)
    table, n = pages_for([(k, k) for k in lens], page, 9, 1)
    cache = gsi.PagedCache(*(torch.randn(n, hkv, page, D, device="cuda", generator=g, dtype=BF) for _ in range(2)))
    q_start = np.cumsum([0] + lens)
    ws = gsi.new_workspace(gsi.paged_attention_workspace_size(cache, hq))
    for _ in range(12):
        Q = 2 * torch.randn(int(q_start[-1]), hq, D, device="cuda", generator=g, dtype=BF)
        first = None
        for _ in range(8):
            out = gsi.paged_attention(cache, Q, i32(q_start), i32(lens), i32(table), max_q=max(lens), workspace=ws)
            first = out if first is None else first
            assert torch.equal(out, first)
        assert gsi.workspace_status(ws) == 0
    for r, k in enumerate(lens):  # the last ones, against the definition
        pg = torch.tensor(table[r, :-(-k // page)], device="cuda").long()
        hidden = torch.ones(k, k, dtype=torch.bool, device="cuda").triu(1)
        for h in (0, 13, 63):
            ks, vs = (t[pg, h // 8].reshape(-1, D)[:k].double() for t in (cache.K, cache.V))
            p = torch.softmax((Q[q_start[r]:q_start[r + 1], h].double() @ ks.T * D ** -0.5).masked_fill(hidden, -float("inf")), -1)
            want, A = p @ vs, p @ vs.abs()
            got = out[q_start[r]:q_start[r + 1], h].double()
            assert ((got - want).abs() <= 1e-4 * A + 2**-8 * (A + want.abs())).all()


def test_attention_offsets_beyond_32_bits(gsi):
    # a cache of more than 2^31 elements, the request's pages at its far end and at its beginning
    hkv, D, page, k = 8, 128, 64, 300
    n_pages = 2**31 // (hkv * D * page) + 40
    K, V = (torch.empty(n_pages, hkv, page, D, dtype=BF, device="cuda") for _ in range(2))
    table = np.array([[n_pages - 1, 0, n_pages - 7, n_pages - 2, 3]], dtype=np.int32)
    small = torch.randn(2, 5, hkv, page, D, device="cuda").to(BF)
    for i, pg in enumerate(table[0]):
        K[pg], V[pg] = small[0, i], small[1, i]
    order = np.arange(5, dtype=np.int32)[None]
    for q in (1, 130):
        Q = torch.randn(q, 16, D, device="cuda").to(BF)
        a = gsi.paged_attention(gsi.PagedCache(K, V), Q, i32([0, q]), i32([k]), i32(table))
        b = gsi.paged_attention(gsi.PagedCache(small[0], small[1]), Q, i32([0, q]), i32([k]), i32(order))
        assert torch.equal(a, b)
    rows = torch.randn(1, (16 + 2 * hkv) * D, device="cuda")
    gsi.cache_append(gsi.PagedCache(K, V), rows, torch.tensor([n_pages * page - 1], device="cuda"), 16)
    assert torch.equal(K[-1, :, -1], rows[0, 16 * D:24 * D].view(hkv, D).to(BF))


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 256), (F, 64)])
@pytest.mark.parametrize("lens", [[(1, 4000), (1, 90)], [(300, 900), (20, 50)]], ids=str)
def test_attention_is_reproducible_and_keeps_its_workspace(gsi, dt, D, lens):
    cache = gsi.PagedCache.empty(1, 2, 16, D, dt)
    ws = gsi.new_workspace(gsi.paged_attention_workspace_size(cache, 4))
    first = None
    for i in range(4):
        out, _ = attention_case(gsi, dt, 4, 2, D, 16, lens, workspace=ws)
        first = out if first is None else first
        assert torch.equal(out, first)
        attention_case(gsi, dt, 4, 2, D, 16, [(1 + 37 * i, 200 + 100 * i)], workspace=ws, seed=i)  # other work between
    assert gsi.workspace_status(ws) == 0


def test_attention_on_another_stream_and_in_a_graph(gsi):
    K, V = (torch.randn(8, 2, 16, 64, device="cuda").to(BF) for _ in range(2))
    cache, Q = gsi.PagedCache(K, V), torch.randn(5, 4, 64, device="cuda").to(BF)
    args = (i32([0, 2, 5]), i32([40, 60]), i32([[0, 1, 2, 7], [3, 4, 5, 6]]))
    want = gsi.paged_attention(cache, Q, *args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gsi.paged_attention(cache, Q, *args, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws, out = gsi.new_workspace(gsi.paged_attention_workspace_size(cache, 4)), torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gsi.paged_attention(cache, Q, *args, out=out, workspace=ws)
    Q2 = torch.randn(5, 4, 64, device="cuda").to(BF)
    Q.copy_(Q2)
    graph.replay()
    graph.replay()
    assert torch.equal(out, gsi.paged_attention(cache, Q2, *args))


def test_attention_of_nothing(gsi):
    cache = gsi.PagedCache.empty(2, 2, 16, 64)
    out = gsi.paged_attention(cache, torch.empty(0, 4, 64, dtype=BF, device="cuda"), i32([0, 0]), i32([5]), i32([[0]]))
    assert out.shape == (0, 4, 64)
    q = torch.ones(2, 4, 64, dtype=BF, device="cuda")
    out = torch.full_like(q, 3.0)
    gsi.paged_attention(cache, q, i32([0]), i32([]), torch.empty(0, 1, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 3.0).all()
    none = gsi.PagedCache.empty(0, 2, 16, 64)
    gsi.paged_attention(none, q, i32([0, 2]), i32([0]), torch.empty(1, 0, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 0.0).all()


@pytest.mark.parametrize("dt,group", [(BF, 8), (BF, 9), (BF, 16), (BF, 128), (F, 16), (F, 17), (F, 32), (F, 64), (F, 65)])
def test_attention_any_hint(gsi, dt, group):
    # no token, one, all of them and no bound: the hint chooses a kernel that holds a token's heads, or none would
    for lens in ([(1, 70), (1, 9)], [(3, 40), (0, 8), (2, 2)]):
        for max_q in (0, 1, sum(q for q, _ in lens), 2**62, 2**63 - 1):
            attention_case(gsi, dt, 2 * group, 2, 64, 16, lens, max_q=max_q)


@pytest.mark.parametrize("dt,hq", [(BF, 4), (BF, 32), (F, 4), (F, 130)])
def test_one_row_of_any_stride(gsi, dt, hq):
    # a view of one row: its stride, that of a matrix of odd width, is never used
    cache = gsi.PagedCache(*(torch.randn(3, 2, 16, 32, device="cuda").to(dt) for _ in range(2)))
    wide = torch.randn((hq + 4) * 32 + 3, device="cuda")
    rows = wide.as_strided((1, (hq + 4) * 32), ((hq + 4) * 32 + 3, 1))
    slots = torch.tensor([20], device="cuda")
    Q = gsi.cache_append(cache, rows, slots, hq)
    assert torch.equal(cache.K[1, :, 4], rows[0, hq * 32:(hq + 2) * 32].view(2, 32).to(dt))
    args = i32([0, 1]), i32([40]), i32([[2, 1, 0]])
    odd = torch.empty(hq * 32 + 1, dtype=dt, device="cuda")[:hq * 32].copy_(Q.view(-1)).as_strided((1, hq, 32), (hq * 32 + 1, 32, 1))
    assert torch.equal(gsi.paged_attention(cache, odd, *args), gsi.paged_attention(cache, Q, *args))


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,d", [(1, 8), (3, 256), (5, 4096), (2, 5120), (17, 1032), (3, 16384), (2, 8200),
                                 (153, 5120), (340, 1032), (170, 5128), (160, 8192), (700, 64)])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "layer"), (None, "rms"), ("rms", None)])
@pytest.mark.parametrize("gate", [None, "row", "index"])
@pytest.mark.parametrize("hdt,ydt,xdt", [(F, F, BF), (BF, F, BF), (F, BF, F), (BF, BF, F)])
def test_norm(gsi, T, d, post, pre, gate, hdt, ydt, xdt):
    g = torch.Generator(device="cuda").manual_seed(d + T)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    h, y = (r(T, d) + 0.5).to(hdt), (2 * r(T, d) - 3.0).to(ydt)
    w = [1 + 0.2 * r(d), r(d), 1 + 0.2 * r(d), r(d)]
    gates = None if gate is None else r(d) if gate == "row" else r(3, d)
    index = i32([(2 * t) % 4 for t in range(T)]) if gate == "index" else None  # index 3 does not exist: a gate of 0

    def make(kind, weight, bias):
        return None if kind is None else gsi.Norm(kind, weight, bias, 1e-5)

    def plain(kind, weight, bias):
        return None if kind is None else (kind, f64(weight), f64(bias), 1e-5)

    ho, x = gsi.norm_residual(h, y, post=make(post, w[0], w[1]), pre=make(pre, w[2], w[3]), gate=gates,
                              gate_index=index, alpha=0.75, x_dtype=xdt)
    H, X = so.norm_residual(f64(h), f64(y), 0.75, plain(post, w[0], w[1]),
                            None if gates is None else f64(gates).reshape(-1, d),
                            None if index is None else index.tolist(), plain(pre, w[2], w[3]))
    for got, want in ((ho, H), (x, X)):
        tol = 2e-5 * (1 + np.abs(want)) + (2**-8 * np.abs(want) if got.dtype == BF else 0)
        assert (np.abs(f64(got) - want) <= tol).all()
    assert ho.dtype == hdt and x.dtype == xdt


@pytest.mark.parametrize("T,d,hdt,ydt,xdt", [(1500, 5120, F, F, BF), (1500, 5120, BF, BF, F), (1525, 4104, F, BF, BF), (27400, 64, F, F, F),
                                             (4000, 1032, BF, F, BF), (1400, 5128, BF, F, BF), (1400, 5128, F, F, F),
                                             (1400, 8192, BF, BF, BF)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["row", "index"])
def test_norm_many_rows_a_cta(gsi, T, d, hdt, ydt, xdt, kind, gate):
    # CTAs that stay copy three rows ahead into a ring of four: nine rows and more of each, so that every slot is filled
    # and read again, with the weights in registers and, above 5120 values, in shared memory; the residual in place
    g = torch.Generator(device="cuda").manual_seed(d + T)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    h, y = (r(T, d) + 0.5).to(hdt), (2 * r(T, d) - 3.0).to(ydt)
    w, b = [1 + 0.2 * r(d), 1 + 0.2 * r(d)], [None, None] if kind == "rms" else [r(d), r(d)]
    gates = r(d) if gate == "row" else r(T // 7, d)
    index = None if gate == "row" else torch.randint(-1, T // 7 + 1, (T,), device="cuda", generator=g).int()
    H, X = so.norm_residual(f64(h), f64(y), 0.75, (kind, f64(w[0]), None if b[0] is None else f64(b[0]), 1e-5),
                            f64(gates).reshape(-1, d), None if index is None else index.tolist(),
                            (kind, f64(w[1]), None if b[1] is None else f64(b[1]), 1e-5))
    ho, x = gsi.norm_residual(h, y, post=gsi.Norm(kind, w[0], b[0]), pre=gsi.Norm(kind, w[1], b[1]), gate=gates, gate_index=index,
                              alpha=0.75, h_out=h, x_dtype=xdt)
    assert ho.data_ptr() == h.data_ptr()
    for got, want in ((ho, H), (x, X)):
        tol = 2e-5 * (1 + np.abs(want)) + (2**-8 * np.abs(want) if got.dtype == BF else 0)
        assert (np.abs(f64(got) - want) <= tol).all()


@pytest.mark.parametrize("T,d", [(1, 8), (3, 1032), (2, 4096), (2, 8200), (700, 64), (340, 1032), (170, 5128), (160, 8192)])
@pytest.mark.parametrize("from_gate", [False, True])
def test_norm_infinity_stays_in_its_column(gsi, T, d, from_gate):
    # an infinite bias or gate of the first column: an RMS norm of the row is 0 elsewhere, whatever the row's length leaves
    # of the last threads without a value
    h, y = torch.randn(T, d, device="cuda"), torch.rand(T, d, device="cuda") + 1
    w, b, gate = torch.ones(d, device="cuda"), torch.randn(d, device="cuda"), torch.ones(d, device="cuda")
    bad = b.clone()
    (gate if from_gate else bad)[0] = float("inf")
    post = None if from_gate else gsi.Norm("rms", w, bad)
    ho, x = gsi.norm_residual(h, y, post=post, gate=gate, pre=gsi.Norm("rms", w, b), x_dtype=F)
    with np.errstate(all="ignore"):
        H, X = so.norm_residual(f64(h), f64(y), 1.0, ("rms", f64(w), f64(bad)) if post else None, f64(gate)[None], None,
                                ("rms", f64(w), f64(b)))
    assert np.isinf(H[:, 0]).all() and np.isnan(X[:, 0]).all() and np.isfinite(X[:, 1:]).all()
    for got, want in ((ho, H), (x, X)):
        assert np.allclose(f64(got), want, rtol=2e-5, atol=2e-5, equal_nan=True)


def test_norm_forms(gsi):
    h = torch.randn(4, 512, device="cuda")
    w = torch.rand(512, device="cuda")
    # the first norm of a model: no block before it
    ho, x = gsi.norm_residual(h, pre=gsi.Norm("rms", w), x_dtype=F)
    assert torch.equal(ho, h)
    assert np.abs(f64(x) - so.norm(f64(h), "rms", f64(w))).max() < 2e-5 * 4
    # in place
    y, keep = torch.randn(4, 512, device="cuda"), h.clone()
    ho, _ = gsi.norm_residual(h, y, pre=gsi.Norm("layer"), alpha=2.0, h_out=h)
    assert ho.data_ptr() == h.data_ptr() and torch.equal(h, 2 * keep + y)
    # nothing to do, and a row of zeros
    assert gsi.norm_residual(h[:0], y[:0], pre=gsi.Norm("rms"))[1].shape == (0, 512)
    _, x = gsi.norm_residual(torch.zeros(1, 512, device="cuda"), pre=gsi.Norm("layer", None, w))
    assert torch.equal(x[0], w.to(BF))
    _, x = gsi.norm_residual(torch.full((1, 512), float("nan"), device="cuda"), pre=gsi.Norm("rms"))
    assert torch.isnan(x.float()).all()


# ------------------------------------------------------------------ refusals
def test_refusals(gsi):
    cache = gsi.PagedCache.empty(4, 2, 16, 64)
    q, st, ln, tb = torch.zeros(2, 4, 64, dtype=BF, device="cuda"), i32([0, 2]), i32([9]), i32([[0]])
    with pytest.raises(ValueError):
        gsi.paged_attention(cache, q.float(), st, ln, tb)
    with pytest.raises(ValueError):
        gsi.paged_attention(cache, q, st.long(), ln, tb)
    with pytest.raises(ValueError):
        gsi.paged_attention(cache, q, st, ln, i32([[0], [1]]))
    with pytest.raises(ValueError):
        gsi.paged_attention(cache, q, st, ln, tb, out=q.float())
    with pytest.raises(gsi.GsiError):
        gsi.paged_attention(cache, q[:, :3].contiguous(), st, ln, tb)
    with pytest.raises(gsi.GsiError):
        gsi.paged_attention(cache, q, st, ln, tb, window=3, causal=False)
    with pytest.raises(gsi.GsiError):
        gsi.paged_attention(cache, q, st, ln, tb, scale=float("inf"))
    with pytest.raises(gsi.GsiError):
        gsi.paged_attention(cache, q, st, ln, tb, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gsi.PagedCache(cache.K, cache.V.permute(0, 2, 1, 3)).desc()
    with pytest.raises(ValueError):
        gsi.paged_attention(gsi.PagedCache(cache.K.cpu(), cache.V.cpu()), q, st, ln, tb)
    with pytest.raises(gsi.GsiError):
        gsi.paged_attention(gsi.PagedCache.empty(4, 2, 24, 64), q, st, ln, tb)
    with pytest.raises(ValueError):
        gsi.cache_append(cache, torch.zeros(2, 8 * 64 + 1, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), 4)
    with pytest.raises(ValueError):
        gsi.cache_append(cache, torch.zeros(2, 8 * 64, device="cuda"), i32([0, 1]), 4)
    with pytest.raises(ValueError):
        gsi.paged_plan(ln, ln, i32([[0], [0]]), tb.view(-1), i32([1]), 16, 4)
    lens = i32([9])
    plan = gsi.PagedPlan.empty(1, 4)
    plan.kv_len = lens
    with pytest.raises(gsi.GsiError):
        gsi.paged_plan(lens, i32([1]), tb, tb.view(-1), i32([1]), 16, plan=plan)
    h = torch.zeros(2, 64, device="cuda")
    with pytest.raises(gsi.GsiError):
        gsi.norm_residual(torch.zeros(2, 12, device="cuda"), pre=gsi.Norm("rms"))
    with pytest.raises(ValueError):
        gsi.norm_residual(h, h, gate=torch.ones(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        gsi.norm_residual(h, pre=gsi.Norm("rms", torch.ones(63, device="cuda")))
    with pytest.raises(gsi.GsiError):
        gsi.norm_residual(h, pre=gsi.Norm("rms", eps=-1.0))
    with pytest.raises(gsi.GsiError):
        gsi.norm_residual(h, alpha=float("nan"))
