"""Serving entry points without a GPU: refusals come before any device call
(fake device pointers, or the injected fault, stop every call here)."""
import ctypes

import pytest
import torch

import __graft_entry__

__graft_entry__.build()
import gated_rank_subspace_gb300 as gsi  # noqa: E402

L = gsi.lib()
P = 0x10000
INF, NAN = float("inf"), float("nan")


def cache(n_pages=8, page=16, heads=2, dim=64, dt=1, ps=None, hs=None, ts=None, K=P, V=P):
    return gsi.CacheDesc(n_pages, page, heads, dim, dt, heads * page * dim if ps is None else ps,
                         page * dim if hs is None else hs, dim if ts is None else ts, K, V)


def attention(c=None, Q=P, q_stride=256, N=4, hq=4, qs=P, ln=P, tb=P, width=3, R=2, max_q=4, scale=0.1, causal=1,
              window=0, O=P, ws=P, n=1 << 30):
    c = cache() if c is None else c
    return L.gsi_paged_attention(ctypes.byref(c), Q, q_stride, N, hq, qs, ln, tb, width, R, max_q, scale, causal, window,
                                 O, ws, n, None)


def plan(cached=P, fresh=P + 16, R=2, tb=P, width=3, free=P, cap=9, nf=P, page=16, N=4, qs=P, ln=P + 32, sl=P, rq=P,
         ps=P, nfo=P + 4, st=P):
    return L.gsi_paged_plan(cached, fresh, R, tb, width, free, cap, nf, page, N, qs, ln, sl, rq, ps, nfo, st, None)


def append(c=None, X=P, xdt=0, stride=512, sl=P, T=4, hq=4, Q=P):
    c = cache() if c is None else c
    return L.gsi_cache_append(ctypes.byref(c), X, xdt, stride, sl, T, hq, Q, None)


def norm(H=P, hdt=0, Y=P, ydt=0, T=2, d=64, alpha=1.0, post=None, gate=None, rows=1, index=None, pre=None, Ho=P, X=P,
         xdt=1):
    b = lambda n: None if n is None else ctypes.byref(n)  # noqa: E731
    return L.gsi_norm_residual(H, hdt, Y, ydt, T, d, alpha, b(post), gate, rows, index, b(pre), Ho, X, xdt, None)


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
    reaches_launch(attention)
    reaches_launch(attention, c=cache(dt=0), q_stride=300)
    reaches_launch(attention, width=0, tb=None)
    reaches_launch(plan)
    reaches_launch(plan, R=0, cached=None, fresh=None, ln=None, tb=None)
    reaches_launch(append)
    reaches_launch(append, Q=None)
    reaches_launch(norm)
    reaches_launch(norm, Y=None, X=None)
    reaches_launch(norm, gate=P, index=P, rows=3, post=gsi.NormDesc(1, 1e-5, P, None))


def test_nothing_to_do_is_no_launch():
    assert attention(N=0, Q=None) == 0 and attention(R=0, qs=None) == 0
    assert append(T=0, X=None) == 0 and norm(T=0, H=None) == 0


@pytest.mark.parametrize("kw,status,needle", [
    (dict(page=24), 2, "page_size"), (dict(page=8), 2, "page_size"), (dict(page=512), 2, "page_size"),
    (dict(dim=260), 2, "head_dim"), (dict(dim=62), 2, "head_dim"), (dict(dim=0), 1, "positive"),
    (dict(dt=5), 1, "dtype"), (dict(ts=60), 2, "stride"), (dict(hs=-64), 1, "stride"), (dict(hs=0), 1, "stride"), (dict(ps=0), 1, "stride"), (dict(K=None), 1, "K is NULL"),
    (dict(V=P + 8), 1, "aligned"), (dict(n_pages=-1), 1, "positive"), (dict(n_pages=1 << 31), 2, "pages"),
    (dict(ps=1 << 40), 2, "stride")])
def test_cache_refusals(kw, status, needle):
    refused(attention(c=cache(**kw)), status, needle)
    refused(append(c=cache(**kw)), status, needle)
    assert L.gsi_paged_attention_workspace_size(ctypes.byref(cache(**kw)), 4) == 0


@pytest.mark.parametrize("kw,status,needle", [
    (dict(N=-1), 1, "negative"), (dict(hq=3), 1, "multiple"), (dict(hq=0), 1, "multiple"), (dict(hq=258, q_stride=258 * 64), 2, "128"),
    (dict(scale=INF), 1, "scale"), (dict(scale=NAN), 1, "scale"), (dict(window=-1), 1, "window"),
    (dict(window=4, causal=0), 1, "window"), (dict(q_stride=255), 1, "q_stride"), (dict(q_stride=260), 2, "q_stride"),
    (dict(Q=None), 1, "Q is NULL"), (dict(O=P + 4), 1, "aligned"), (dict(qs=None), 1, "q_start"), (dict(tb=None), 1, "table"),
    (dict(ws=None), 4, "NULL"), (dict(ws=P + 16), 4, "256-byte"), (dict(n=8), 4, "needed"), (dict(N=1 << 25), 2, "2^24"),
    (dict(width=1 << 28), 2, "2^31"), (dict(width=(1 << 27) - 31), 2, "2^31"), (dict(ln=P + 2), 1, "aligned")])
def test_attention_refusals(kw, status, needle):
    refused(attention(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(R=-1), 1, "negative"), (dict(page=20), 2, "page_size"), (dict(ln=P, cached=P), 1, "kv_len"),
    (dict(nfo=P), 1, "n_free"), (dict(N=1 << 25), 2, "2^24"), (dict(R=1 << 21), 2, "2^20"), (dict(sl=P + 4), 1, "slots"),
    (dict(free=None), 1, "free_pages"), (dict(st=None), 1, "status"), (dict(fresh=None), 1, "fresh"),
    (dict(width=1 << 28), 2, "2^31")])
def test_plan_refusals(kw, status, needle):
    refused(plan(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), 1, "negative"), (dict(hq=-1), 1, "negative"), (dict(stride=500), 1, "row_stride"), (dict(stride=514), 2, "row_stride"),
    (dict(X=None), 1, "X is NULL"), (dict(sl=P + 4), 1, "slots"), (dict(Q=P + 2), 1, "Q is not"), (dict(xdt=3), 1, "dtype")])
def test_append_refusals(kw, status, needle):
    refused(append(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(d=12), 2, "multiple of 8"), (dict(d=16392), 2, "16384"), (dict(d=0), 1, "positive"), (dict(T=-1), 1, "positive"),
    (dict(alpha=NAN), 1, "alpha"), (dict(H=None), 1, "H is NULL"), (dict(Ho=None, X=None), 1, "both NULL"),
    (dict(post=gsi.NormDesc(3, 1e-5, None, None)), 1, "unknown norm"), (dict(pre=gsi.NormDesc(1, -1.0, None, None)), 1, "eps"),
    (dict(pre=gsi.NormDesc(1, NAN, None, None)), 1, "eps"), (dict(pre=gsi.NormDesc(1, 0.0, P + 4, None)), 1, "aligned"),
    (dict(gate=P, rows=0), 1, "gate_rows"), (dict(gate=P + 8), 1, "aligned"), (dict(hdt=9), 1, "dtype")])
def test_norm_refusals(kw, status, needle):
    refused(norm(**kw), status, needle)


def test_workspace_size_is_host_arithmetic():
    for kw in (dict(), dict(dim=256), dict(dt=0), dict(dim=80)):
        n = L.gsi_paged_attention_workspace_size(ctypes.byref(cache(**kw)), 4)
        assert 256 <= n <= 96 << 20 and n % 256 == 0
    assert L.gsi_paged_attention_workspace_size(ctypes.byref(cache()), 3) == 0


# ------------------------------------------------------------------ devices
class On:
    """A tensor that says it lies on a GPU (its data is never read: the injected fault stops every call)."""

    def __init__(self, device, *shape, dtype=torch.int32):
        self.t, self.device_no = torch.zeros(*shape, dtype=dtype), device

    def __getattr__(self, name):
        return getattr(self.t, name)

    is_cuda = property(lambda self: self.device_no >= 0)
    device = property(lambda self: torch.device("cuda", self.device_no) if self.device_no >= 0 else torch.device("cpu"))

    def get_device(self):
        return self.device_no

    def data_ptr(self):
        return P if self.t.numel() else 0


@pytest.fixture
def current(monkeypatch):
    """Makes a device current."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    return lambda device: monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: device, raising=False)


BF, I64 = torch.bfloat16, torch.int64
SHAPES = {
    "plan": dict(cached=(2,), fresh=(2,), table=(2, 3), free=(9,), n_free=(1,), q_start=(3,), kv_len=(2,), slots=(4, I64),
                 token_req=(4,), positions=(4,), left=(1,), status=(1,)),
    "append": dict(K=(8, 2, 16, 64, BF), V=(8, 2, 16, 64, BF), rows=(4, 512, torch.float32), slots=(4, I64), Q=(4, 4, 64, BF)),
    "attention": dict(K=(8, 2, 16, 64, BF), V=(8, 2, 16, 64, BF), Q=(4, 4, 64, BF), q_start=(3,), kv_len=(2,), table=(2, 3),
                      out=(4, 4, 64, BF), workspace=(64 << 20, torch.uint8)),
    "norm": dict(h=(4, 64, torch.float32), y=(4, 64, torch.float32), w0=(64, torch.float32), b0=(64, torch.float32),
                 w1=(64, torch.float32), b1=(64, torch.float32), gate=(3, 64, torch.float32), index=(4,),
                 h_out=(4, 64, torch.float32), x=(4, 64, BF)),
}


def call(op, t):
    if op == "plan":
        plan = gsi.PagedPlan(t["q_start"], t["kv_len"], t["slots"], t["token_req"], t["positions"], t["left"], t["status"])
        plan.kv_len.data_ptr = plan.n_free.data_ptr = lambda: P + 64
        gsi.paged_plan(t["cached"], t["fresh"], t["table"], t["free"], t["n_free"], 16, plan=plan)
    elif op == "append":
        gsi.cache_append(gsi.PagedCache(t["K"], t["V"]), t["rows"], t["slots"], 4, Q=t["Q"])
    elif op == "attention":
        gsi.paged_attention(gsi.PagedCache(t["K"], t["V"]), t["Q"], t["q_start"], t["kv_len"], t["table"], out=t["out"],
                            workspace=t["workspace"])
    else:
        gsi.norm_residual(t["h"], t["y"], post=gsi.Norm("layer", t["w0"], t["b0"]), pre=gsi.Norm("layer", t["w1"], t["b1"]),
                          gate=t["gate"], gate_index=t["index"], h_out=t["h_out"], x=t["x"])


def tensors(op, device):
    made = {}
    for name, shape in SHAPES[op].items():
        dtype = shape[-1] if isinstance(shape[-1], torch.dtype) else torch.int32
        made[name] = On(device, *(s for s in shape if not isinstance(s, torch.dtype)), dtype=dtype)
    return made


@pytest.mark.parametrize("op,name,elsewhere", [(op, name, d) for op in SHAPES for name in [None, *SHAPES[op]]
                                               for d in ([1] if name is None else [1, -1])])
def test_tensors_lie_on_the_current_device(current, op, name, elsewhere):
    # a kernel runs on the device that is current: pointers of another one, or of the host, would fault there
    made = tensors(op, 0)
    L.gsi_debug_fail_after(1)
    try:
        current(0)
        if name is None:
            with pytest.raises(gsi.GsiError, match="injected"):  # all on the current device: reaches the launch
                call(op, made)
            L.gsi_debug_fail_after(1)
            current(elsewhere)
            with pytest.raises(ValueError, match="device"):
                call(op, made)
        else:
            made[name].device_no = elsewhere
            with pytest.raises(ValueError):
                call(op, made)
    finally:
        L.gsi_debug_fail_after(0)


def test_a_gate_of_no_rows_is_not_no_gate(current):
    # an empty tensor has no address, which to the library is "no gate": a gate of 1, where no index is right
    current(0)
    made = tensors("norm", 0)
    made["gate"] = On(0, 0, 64, dtype=torch.float32)
    L.gsi_debug_fail_after(1)
    try:
        with pytest.raises(ValueError, match="gate"):
            call("norm", made)
    finally:
        L.gsi_debug_fail_after(0)
    # no tokens ask for no rows
    for name, shape in SHAPES["norm"].items():
        if shape[0] == 4:
            made[name] = On(0, 0, *(s for s in shape[1:-1]), dtype=shape[-1]) if len(shape) > 1 else On(0, 0)
    call("norm", made)


def test_the_stride_of_one_row_means_nothing():
    # a single row has no next one: whatever its stride says, as of a view's row
    for stride in (0, 1, 513, -8, 1 << 40):
        reaches_launch(append, T=1, stride=stride)
        reaches_launch(attention, N=1, q_stride=stride)
        reaches_launch(attention, c=cache(dt=0), N=1, q_stride=stride)


@pytest.mark.parametrize("heads,needle", [(3, "multiple"), (0, "multiple"), (-2, "multiple"), (258, "128"), (2 << 32, "128")])
def test_workspace_of_a_refused_shape_says_why(heads, needle):
    attention(scale=NAN)  # an earlier error is not this one
    n = L.gsi_paged_attention_workspace_size(ctypes.byref(cache()), heads)
    refused(1 if n == 0 else 0, 1, needle)
    assert L.gsi_paged_attention_workspace_size(ctypes.byref(cache()), 4) > 0 and L.gsi_last_error() == b""
