"""Entry points for long contexts and drafted tokens without a GPU: refusals come
before any device call (fake device pointers, or the injected fault, stop every
call here), and the angles' table is made on the host."""
import ctypes
import math
import random
from decimal import Decimal, getcontext

import pytest
import torch

import __graft_entry__

__graft_entry__.build()
import gated_rank_subspace_gb300 as gsi  # noqa: E402
from oracle import context_oracle as co  # noqa: E402

L = gsi.lib()
P = 0x10000
INF, NAN = float("inf"), float("nan")


def cache(n_pages=8, page=16, heads=2, dim=64, dt=1, ps=None, hs=None, ts=None, K=P, V=P):
    return gsi.CacheDesc(n_pages, page, heads, dim, dt, heads * page * dim if ps is None else ps,
                         page * dim if hs is None else hs, dim if ts is None else ts, K, V)


def turn(dim=32, layout=0, scale=1.0, phases=P):
    return gsi.RotaryDesc(dim, layout, scale, phases)


def rotary(c=None, X=P, xdt=0, stride=512, sl=P, pos=P, req=P, off=P, R=2, T=4, hq=4, rot=..., Q=P):
    c, rot = cache() if c is None else c, turn() if rot is ... else rot
    return L.gsi_rotary_append(ctypes.byref(c), X, xdt, stride, sl, pos, req, off, R, T, hq, None if rot is None else ctypes.byref(rot), Q, None)


def attention(c=None, lse=P, **kw):
    c = cache() if c is None else c
    return L.gsi_paged_attention_lse(ctypes.byref(c), P, 256, 4, 4, P, P, P, 3, 2, 4, 0.1, 1, 0, P, lse, P, 1 << 30, None)


def weights(c=None, Q=P, q_stride=256, N=4, hq=4, lse=P, qs=P, ln=P, held=P, off=P, tb=P, width=3, R=2, max_q=4, scale=0.1, causal=1,
            marks=..., ws=P, n=1 << 30):
    c, marks = cache() if c is None else c, gsi.MarksDesc(P, P) if marks is ... else marks
    return L.gsi_key_weights(ctypes.byref(c), Q, q_stride, N, hq, lse, qs, ln, held, off, tb, width, R, max_q, scale, causal,
                             None if marks is None else ctypes.byref(marks), ws, n, None)


def evict(c=None, ln=P, tb=P, width=3, R=2, marks=..., budget=8, recent=2, sinks=1, off=P + 16, kept=P + 32, out=P + 48, ws=P, n=1 << 30):
    c, marks = cache() if c is None else c, gsi.MarksDesc(P, P) if marks is ... else marks
    return L.gsi_cache_evict(ctypes.byref(c), ln, tb, width, R, None if marks is None else ctypes.byref(marks), budget, recent, sinks, off,
                             kept, out, ws, n, None)


def verify(target=P, tdt=0, ts=100, draft=P, ddt=0, ds=100, N=4, V=100, tok=P, u=P, v=P, qs=P, ln=P, R=2, out=P + 64, acc=P + 16, kept=P + 32):
    return L.gsi_verify_drafts(target, tdt, ts, draft, ddt, ds, N, V, tok, u, v, qs, ln, R, out, acc, kept, None)


def trim(ln=P, kept=P, R=2, tb=P, width=3, free=P, cap=9, nf=P, page=16, nfo=P + 4, st=P):
    return L.gsi_paged_trim(ln, kept, R, tb, width, free, cap, nf, page, nfo, st, None)


def refused(status, want, needle):
    assert status == want
    assert needle in L.gsi_last_error().decode()


def reaches_launch(call, **kw):
    L.gsi_debug_fail_after(1)
    try:
        refused(call(**kw), 3, "injected")
    finally:
        L.gsi_debug_fail_after(0)


def test_what_is_valid_reaches_the_launch():
    for call in (rotary, attention, weights, evict, verify, trim):
        reaches_launch(call)
    reaches_launch(attention, lse=None)
    reaches_launch(rotary, Q=None, req=None, off=None, R=0)
    reaches_launch(rotary, T=1, stride=0)
    reaches_launch(rotary, rot=turn(dim=64, layout=1))
    reaches_launch(weights, held=None, off=None)
    reaches_launch(weights, N=0, Q=None, lse=None)
    reaches_launch(weights, N=1, q_stride=0)
    reaches_launch(evict, off=None, out=None)
    reaches_launch(evict, budget=3, recent=2, sinks=1)
    reaches_launch(verify, draft=None, ds=0, ddt=9)
    reaches_launch(verify, ln=None, kept=None)
    reaches_launch(verify, kept=P, ln=P)
    reaches_launch(verify, target=P + 2, tdt=1, ts=101)
    reaches_launch(verify, N=0, target=None, draft=None, tok=None, u=None, v=None, out=None)
    reaches_launch(trim, R=0, ln=None, kept=None, tb=None)


def test_nothing_to_do_is_no_launch():
    assert rotary(T=0, X=None, sl=None, pos=None) == 0
    assert weights(R=0, qs=None, ln=None, tb=None) == 0 and weights(width=0, tb=None) == 0
    assert weights(c=cache(n_pages=0, K=None, V=None), marks=gsi.MarksDesc(None, None)) == 0
    assert evict(R=0, ln=None, tb=None, kept=None) == 0 and verify(R=0, qs=None) == 0


@pytest.mark.parametrize("call", [rotary, weights, evict])
@pytest.mark.parametrize("kw,status,needle", [(dict(page=24), 2, "page_size"), (dict(dim=260), 2, "head_dim"), (dict(dim=62), 2, "head_dim"),
                                              (dict(dt=5), 1, "dtype"), (dict(ts=60), 2, "stride"), (dict(hs=0), 1, "stride"),
                                              (dict(K=None), 1, "K is NULL"), (dict(V=P + 8), 1, "aligned")])
def test_caches(call, kw, status, needle):
    refused(call(c=cache(**kw)), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rot=None), 1, "rotary"), (dict(rot=turn(dim=0)), 1, "rotary dim"), (dict(rot=turn(dim=31)), 1, "rotary dim"),
    (dict(rot=turn(dim=66)), 1, "rotary dim"), (dict(rot=turn(layout=2)), 1, "layout"), (dict(rot=turn(scale=INF)), 1, "scale"),
    (dict(rot=turn(scale=NAN)), 1, "scale"), (dict(rot=turn(phases=None)), 1, "phases"), (dict(rot=turn(phases=P + 4)), 1, "phases"),
    (dict(pos=None), 1, "positions"), (dict(pos=P + 2), 1, "positions"), (dict(req=P + 1), 1, "aligned"), (dict(off=P + 2), 1, "aligned"),
    (dict(R=-1), 1, "negative"), (dict(R=1 << 21), 2, "2^20"), (dict(X=None), 1, "X is NULL"), (dict(stride=500), 1, "row_stride"),
    (dict(stride=514), 2, "row_stride"), (dict(T=-1), 1, "negative"), (dict(T=(1 << 24) + 1), 2, "2^24"), (dict(xdt=3), 1, "dtype"),
    (dict(sl=P + 4), 1, "slots"), (dict(Q=P + 8), 1, "Q is not")])
def test_rotary_refusals(kw, status, needle):
    refused(rotary(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(hq=3), 1, "n_q_heads"), (dict(hq=258), 2, "128"), (dict(scale=NAN), 1, "scale"), (dict(N=-1), 1, "negative"),
    (dict(N=(1 << 24) + 1), 2, "2^24"), (dict(R=(1 << 20) + 1), 2, "2^20"), (dict(width=1 << 27), 2, "2^31"), (dict(q_stride=248), 1, "q_stride"),
    (dict(q_stride=260), 2, "q_stride"), (dict(q_stride=1 << 38), 2, "q_stride"), (dict(Q=None), 1, "Q is NULL"), (dict(Q=P + 8), 1, "Q is not"),
    (dict(lse=None), 1, "LSE"), (dict(lse=P + 2), 1, "LSE"), (dict(qs=None), 1, "q_start"), (dict(ln=None), 1, "kv_len"),
    (dict(tb=None), 1, "table"), (dict(held=P + 1), 1, "held"), (dict(off=P + 2), 1, "offsets"), (dict(marks=None), 1, "marks"),
    (dict(marks=gsi.MarksDesc(None, P)), 1, "weight"), (dict(marks=gsi.MarksDesc(P, P + 2)), 1, "place"), (dict(ws=None), 4, "workspace"),
    (dict(ws=P + 16), 4, "aligned"), (dict(n=100), 4, "bytes"), (dict(max_q=-1), 1, "negative")])
def test_weights_refusals(kw, status, needle):
    refused(weights(**kw), status, needle)


def test_lse_has_to_be_aligned():
    refused(attention(lse=P + 2), 1, "LSE")


@pytest.mark.parametrize("kw,status,needle", [
    (dict(budget=0), 1, "budget"), (dict(budget=-4), 1, "budget"), (dict(budget=1 << 31), 2, "2^31"), (dict(recent=-1), 1, "recent"),
    (dict(sinks=-1), 1, "sinks"), (dict(recent=8, sinks=1), 1, "within the budget"), (dict(recent=1 << 40), 1, "within the budget"),
    (dict(sinks=1 << 62, recent=8), 1, "within"), (dict(R=-1), 1, "negative"), (dict(R=(1 << 20) + 1), 2, "2^20"),
    (dict(c=cache(heads=4096), R=1 << 16), 2, "2^27"), (dict(width=-1), 1, "negative"), (dict(width=1 << 27), 2, "2^31"),
    (dict(ln=None), 1, "kv_len"), (dict(tb=None), 1, "table"), (dict(kept=None), 1, "kept"), (dict(kept=P), 1, "read"),
    (dict(kept=P + 16), 1, "read"), (dict(out=P), 1, "read"), (dict(out=P + 16), 1, "read"), (dict(out=P + 32), 1, "both are one"),
    (dict(off=P + 2), 1, "aligned"), (dict(out=P + 50), 1, "aligned"), (dict(marks=None), 1, "marks"), (dict(marks=gsi.MarksDesc(P, None)), 1, "place"),
    (dict(ws=None), 4, "workspace"), (dict(ws=P + 64), 4, "aligned"), (dict(n=4608), 4, "needed")])
def test_evict_refusals(kw, status, needle):
    refused(evict(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(tdt=2), 1, "dtype"), (dict(ddt=-1), 1, "dtype"), (dict(N=-1), 1, "sizes"), (dict(R=-1), 1, "sizes"), (dict(V=0), 1, "sizes"),
    (dict(N=(1 << 24) + 1), 2, "2^24"), (dict(R=(1 << 20) + 1), 2, "2^20"), (dict(V=(1 << 24) + 1, ts=1 << 30, ds=1 << 30), 2, "2^24"),
    (dict(ts=99), 1, "stride"), (dict(ds=99), 1, "stride"), (dict(ts=1 << 38), 2, "stride"), (dict(ds=1 << 38), 2, "stride"),
    (dict(target=None), 1, "target"), (dict(target=P + 2), 1, "target"), (dict(draft=P + 1, ddt=1), 1, "draft"), (dict(tok=None), 1, "tokens"),
    (dict(u=None), 1, "uniforms"), (dict(v=None), 1, "samples"), (dict(out=None), 1, "out"), (dict(out=P), 1, "out is tokens"),
    (dict(qs=None), 1, "q_start"), (dict(acc=None), 1, "accepted"), (dict(ln=None), 1, "together"), (dict(kept=None), 1, "together"),
    (dict(acc=P + 32), 1, "accepted is"), (dict(acc=P), 1, "accepted is"), (dict(kept=P + 2), 1, "aligned")])
def test_verify_refusals(kw, status, needle):
    refused(verify(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(page=20), 2, "page_size"), (dict(R=-1), 1, "negative"), (dict(width=-1), 1, "negative"), (dict(cap=-1), 1, "negative"),
    (dict(R=(1 << 20) + 1), 2, "2^20"), (dict(width=1 << 27), 2, "2^31"), (dict(cap=1 << 31), 2, "2^31"), (dict(ln=None), 1, "kv_len"),
    (dict(kept=P + 1), 1, "kept"), (dict(tb=None), 1, "table"), (dict(free=None), 1, "free_pages"), (dict(nf=None), 1, "n_free"),
    (dict(nfo=None), 1, "n_free_out"), (dict(nfo=P), 1, "n_free_out is n_free"), (dict(st=None), 1, "status")])
def test_trim_refusals(kw, status, needle):
    refused(trim(**kw), status, needle)


def test_workspace_sizes():
    c = cache()
    size = L.gsi_cache_evict_workspace_size
    assert size(ctypes.byref(c), 3, 100) >= 3 * 2 * 100 * 8 and size(ctypes.byref(c), 0, 1) > 0
    assert size(ctypes.byref(c), 3, 0) == 0 and "budget" in L.gsi_last_error().decode()
    assert size(ctypes.byref(cache(page=24)), 3, 4) == 0 and "page_size" in L.gsi_last_error().decode()
    assert L.gsi_key_weights_workspace_size() % 256 == 0


# ------------------------------------------------------------------ the angles' table
@pytest.mark.parametrize("dim", [2, 8, 20, 64, 128, 256])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0), dict(base=500000.0),
                                dict(scaling="yarn", factor=16.0, context=4096, fast=32.0, slow=1.0), dict(scaling="yarn", factor=1.0, context=100.0, fast=2.0, slow=1.0),
                                dict(scaling="bands", factor=8.0, context=8192, fast=4.0, slow=1.0), dict(scaling="bands", factor=8.0, context=10.0, fast=4.0, slow=1.0)])
def test_rates(dim, kw):
    if dim == 2 and kw.get("scaling") == "ntk":
        with pytest.raises(gsi.GsiError):
            gsi.Rotary.rates(dim, **kw)
        return
    got, scale = gsi.Rotary.rates(dim, **kw)
    want, s = co.rotary_rates(dim, **kw)
    assert len(got) == dim // 2 and all(abs(a - b) <= 1e-14 * b for a, b in zip(got, want)) and abs(scale - s) <= 2**-23 * s


def test_rates_have_their_ends():
    plain, _ = gsi.Rotary.rates(128)
    ntk, _ = gsi.Rotary.rates(128, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and abs(ntk[-1] * 8 / plain[-1] - 1) < 1e-12
    for scaling in ("yarn", "bands"):
        w, _ = gsi.Rotary.rates(128, scaling=scaling, factor=8.0, context=8192)
        assert w[0] == plain[0] and abs(w[-1] * 8 / plain[-1] - 1) < 1e-12
        assert all(p / 8 - 1e-18 <= x <= p for x, p in zip(w, plain))


@pytest.mark.parametrize("kw,needle", [(dict(dim=0), "dim"), (dict(dim=5), "dim"), (dict(dim=258), "dim"), (dict(base=1.0), "base"),
                                       (dict(base=INF), "base"), (dict(scaling="linear", factor=0.5), "factor"), (dict(scaling="ntk", factor=NAN), "factor"),
                                       (dict(scaling="yarn", factor=2.0), "context"), (dict(scaling="bands", factor=2.0, context=10.0, fast=1.0, slow=2.0), "fast"),
                                       (dict(scaling="bands", factor=2.0, context=10.0, fast=1.0, slow=-1.0), "fast")])
def test_rates_refusals(kw, needle):
    with pytest.raises(gsi.GsiError, match=needle):
        gsi.Rotary.rates(**{"dim": 64, **kw})


def test_phases_are_turns():
    getcontext().prec = 80
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    rng = random.Random(1)
    rates = [1.0, 0.5, 1e-5, 1e-12, 0.0, -1.0, 2 * math.pi, 100.0] + [rng.uniform(0, 1) for _ in range(200)]
    w, out = (ctypes.c_double * len(rates))(*rates), (ctypes.c_uint64 * len(rates))()
    assert L.gsi_rotary_phases(w, len(rates), out) == 0
    for r, p in zip(rates, out):
        exact = Decimal(r) / (2 * pi) % 1 * 2**64
        off = (int(p) - int(exact.to_integral_value())) % 2**64
        # one rounding of the sum's low part and one of the whole, for rates below a turn; 2^-52 of a larger one's turns
        assert min(off, 2**64 - off) <= max(2, abs(r) * 64), r
    assert L.gsi_rotary_phases(w, 0, None) == 0
    refused(L.gsi_rotary_phases(None, 1, out), 1, "rates")
    w[3] = INF
    refused(L.gsi_rotary_phases(w, len(rates), out), 1, "not finite")


def test_python_refusals_without_a_gpu():
    with pytest.raises(gsi.GsiError, match="finite"):
        gsi.Rotary.from_rates([NAN], device="cpu")
    r = gsi.Rotary.from_rates([1.0, 0.5], device="cpu")
    assert r.dim == 4 and r.phases.dtype is torch.int64 and abs(int(r.phases[0]) / 2**64 - 1 / (2 * math.pi)) < 1e-18
    with pytest.raises(ValueError, match="device"):
        gsi.verify_drafts(torch.zeros(1, 3), None, None, None, None, None)
