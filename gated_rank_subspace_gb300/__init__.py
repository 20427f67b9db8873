"""Python binding of libgsi, the gated-subspace linear map on one sm_103a GPU.

The method ("Gated Subspace Inference for Transformer Acceleration",
gist.science technical summary, §2.1-§2.2): for a map W and an orthonormal
basis V_k, each token x is projected, g = V_k^T x; its residual ratio
rho = ||x - V_k g|| / ||x|| decides the path: rho < eps gives the fast path
y = M g with the cached image M = W V_k, otherwise the exact y = W x.

This module only marshals arguments: every step runs in the library's CUDA
kernels (include/gsi.h documents the C ABI).  PyTorch supplies device memory
and streams.  There is no CPU fallback: if libgsi.so has not been built, or
no GPU is present, calls fail loudly.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgsi.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "gsi.h")

GSI_F32, GSI_BF16 = 0, 1
PATHS = {"auto": 0, "stream": 1, "tensor": 2, "fused": 3, "batch": 4}
STATUS = {0: "GSI_OK", 1: "GSI_ERR_INVALID_ARG", 2: "GSI_ERR_UNSUPPORTED", 3: "GSI_ERR_CUDA",
          4: "GSI_ERR_WORKSPACE", 5: "GSI_ERR_TIMEOUT"}


class GsiError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


class MapDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int64), ("d_out", ctypes.c_int64), ("k", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("W", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("M", ctypes.c_void_p), ("gram", ctypes.c_void_p)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("n_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("dtype", ctypes.c_int), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("K", ctypes.c_void_p),
                ("V", ctypes.c_void_p)]


class NormDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int64), ("layout", ctypes.c_int), ("scale", ctypes.c_float), ("phases", ctypes.c_void_p)]


class MarksDesc(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("place", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgsi.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(or python -m gated_rank_subspace_gb300._build)")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, f32, f64, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "gsi_build_image": [vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, vp],
        "gsi_build_image_ex": [vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, vp, sz, vp],
        "gsi_linear_workspace_size": [P(MapDesc), i64, ctypes.c_int, P(sz)],
        "gsi_workspace_init": [vp, sz, vp],
        "gsi_workspace_status": [vp, P(ctypes.c_uint32), vp],
        "gsi_gate": [P(MapDesc), vp, i64, f32, vp, vp, vp, vp, sz, vp],
        "gsi_compact": [vp, i64, vp, vp, vp],
        "gsi_apply": [P(MapDesc), vp, vp, i64, vp, vp, sz, vp],
        "gsi_linear": [P(MapDesc), vp, i64, f32, vp, vp, vp, vp, sz, vp],
        "gsi_linear_ex": [P(MapDesc), vp, i64, f32, vp, vp, vp, vp, sz, ctypes.c_int, vp],
        "gsi_stack_workspace_size": [P(MapDesc), i64, i64, P(sz)],
        "gsi_stack": [P(MapDesc), i64, P(vp), i64, f32, P(vp), P(vp), vp, sz, vp],
        "gsi_stack_ex": [P(MapDesc), i64, P(vp), i64, f32, P(vp), P(vp), vp, sz, ctypes.c_int, vp],
        "gsi_path_errors": [P(MapDesc), vp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "gsi_eps_sweep": [vp, vp, vp, i64, vp, i64, i64, vp, vp, vp, vp],
        "gsi_basis_orthonormalize": [vp, i64, i64, vp, vp],
        "gsi_basis_step": [vp, ctypes.c_int, i64, i64, i64, vp, vp, sz, vp, vp],
        "gsi_basis_coherence": [vp, vp, i64, i64, vp, vp, vp],
        "gsi_basis_export": [vp, i64, i64, vp, ctypes.c_int, vp],
        "gsi_residual_check": [P(MapDesc), vp, i64, vp, vp, vp, vp, vp, sz, vp],
        "gsi_paged_plan": [vp, vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp],
        "gsi_cache_append": [P(CacheDesc), vp, ctypes.c_int, i64, vp, i64, i64, vp, vp],
        "gsi_paged_attention": [P(CacheDesc), vp, i64, i64, i64, vp, vp, vp, i64, i64, i64, f32, ctypes.c_int, i64, vp,
                                vp, sz, vp],
        "gsi_paged_attention_lse": [P(CacheDesc), vp, i64, i64, i64, vp, vp, vp, i64, i64, i64, f32, ctypes.c_int, i64, vp,
                                    vp, vp, sz, vp],
        "gsi_paged_trim": [vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp],
        "gsi_rotary_rates": [i64, f64, ctypes.c_int, f64, f64, f64, f64, P(f64), P(f32)],
        "gsi_rotary_phases": [P(f64), i64, P(ctypes.c_uint64)],
        "gsi_rotary_append": [P(CacheDesc), vp, ctypes.c_int, i64, vp, vp, vp, vp, i64, i64, i64, P(RotaryDesc), vp, vp],
        "gsi_key_weights": [P(CacheDesc), vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, i64, i64, i64, f32, ctypes.c_int,
                            P(MarksDesc), vp, sz, vp],
        "gsi_cache_evict": [P(CacheDesc), vp, vp, i64, i64, P(MarksDesc), i64, i64, i64, vp, vp, vp, vp, sz, vp],
        "gsi_verify_drafts": [vp, ctypes.c_int, i64, vp, ctypes.c_int, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp],
        "gsi_norm_residual": [vp, ctypes.c_int, vp, ctypes.c_int, i64, i64, f32, P(NormDesc), vp, i64, vp, P(NormDesc),
                              vp, vp, ctypes.c_int, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.gsi_build_image_work_bytes.argtypes = [i64, i64, ctypes.c_int]
    L.gsi_build_image_work_bytes.restype = sz
    L.gsi_residual_check_work_bytes.argtypes = [i64, i64]
    L.gsi_residual_check_work_bytes.restype = sz
    L.gsi_basis_step_work_bytes.argtypes = [i64, i64, i64]
    L.gsi_basis_step_work_bytes.restype = sz
    L.gsi_paged_attention_workspace_size.argtypes = [P(CacheDesc), i64]
    L.gsi_paged_attention_workspace_size.restype = sz
    L.gsi_key_weights_workspace_size.argtypes = []
    L.gsi_key_weights_workspace_size.restype = sz
    L.gsi_cache_evict_workspace_size.argtypes = [P(CacheDesc), i64, i64]
    L.gsi_cache_evict_workspace_size.restype = sz
    L.gsi_last_error.argtypes = []
    L.gsi_last_error.restype = ctypes.c_char_p
    L.gsi_debug_fail_after.argtypes = [ctypes.c_int]
    L.gsi_debug_fail_after.restype = None
    L.gsi_debug_withhold_slice.argtypes = [ctypes.c_int]
    L.gsi_debug_withhold_slice.restype = None
    L.gsi_debug_refuse_coresident.argtypes = [ctypes.c_int]
    L.gsi_debug_refuse_coresident.restype = None
    L.gsi_linear_noalloc.argtypes = [P(MapDesc), vp, i64, f32, vp, vp, vp, vp]
    L.gsi_linear_noalloc.restype = ctypes.c_int
    L.gsi_linear_noalloc_max_bytes.argtypes = []
    L.gsi_linear_noalloc_max_bytes.restype = sz
    L.gsi_linear_noalloc_status.argtypes = [P(ctypes.c_uint32), vp]
    L.gsi_linear_noalloc_status.restype = ctypes.c_int
    _lib = L
    return L


def declared_symbols() -> list:
    """Entry points declared in include/gsi.h."""
    src = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(gsi_\w+)\s*\(", src, re.M)))


def _check(status: int):
    if status != 0:
        raise GsiError(status, lib().gsi_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _raw_stream(stream, t):
    """The stream's handle as a number (the current stream of t's device by default)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(t.get_device())  # current_stream(t.device) builds two objects for it


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return GSI_F32
    if dt == torch.bfloat16:
        return GSI_BF16
    raise TypeError(f"unsupported dtype {dt}: float32 or bfloat16")


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


@dataclass
class Map:
    """One linear map with its cached artefacts (device tensors).

    W: d_out x d, V: d x k, M: d_out x k (same dtype), gram: k x k float32.
    """
    W: torch.Tensor
    V: torch.Tensor
    M: torch.Tensor
    gram: torch.Tensor

    @property
    def d(self):
        return self.W.shape[1]

    @property
    def d_out(self):
        return self.W.shape[0]

    @property
    def k(self):
        return self.V.shape[1]

    def desc(self) -> MapDesc:
        return MapDesc(self.d, self.d_out, self.k, _dtype_code(self.W.dtype), self.W.data_ptr(),
                       self.V.data_ptr(), self.M.data_ptr(),
                       self.gram.data_ptr() if self.gram is not None else None)


def build_image(W: torch.Tensor, V: torch.Tensor, M=None, gram=None, with_gram=True, stream=None,
                tensor_cores=True):
    """M = W V (and the Gram V^T V) on the GPU; returns (M, gram).  bf16 maps
    use the tensor cores (a scratch area is allocated here, by PyTorch)
    unless tensor_cores is False, which keeps the CUDA-core kernel."""
    _require_cuda(W, V)
    d_out, d = W.shape
    k = V.shape[1]
    if M is None:
        M = torch.empty(d_out, k, dtype=W.dtype, device=W.device)
    if gram is None and with_gram:
        gram = torch.empty(k, k, dtype=torch.float32, device=W.device)
    dt = _dtype_code(W.dtype)
    nwork = int(lib().gsi_build_image_work_bytes(d, k, dt)) if tensor_cores else 0
    if nwork:
        work = torch.empty(nwork, dtype=torch.uint8, device=W.device)
        _check(lib().gsi_build_image_ex(_ptr(W), _ptr(V), _ptr(M), _ptr(gram), d, d_out, k, dt, _ptr(work),
                                        nwork, _stream(stream)))
        if workspace_status(work, stream) != 0:
            raise GsiError(5, "image build: a bounded device wait gave up")
    else:
        _check(lib().gsi_build_image(_ptr(W), _ptr(V), _ptr(M), _ptr(gram), d, d_out, k, dt, _stream(stream)))
    return M, gram


def make_map(W: torch.Tensor, V: torch.Tensor, stream=None) -> Map:
    """Upload-ready map: builds the image and the Gram on the GPU."""
    M, gram = build_image(W, V, stream=stream)
    return Map(W, V, M, gram)


def workspace_size(m: Map, T: int, path: str = "auto") -> int:
    n = ctypes.c_size_t(0)
    desc = m.desc()
    _check(lib().gsi_linear_workspace_size(ctypes.byref(desc), T, PATHS[path], ctypes.byref(n)))
    return n.value


def stack_workspace_size(maps, T: int) -> int:
    arr = (MapDesc * len(maps))(*[m.desc() for m in maps])
    n = ctypes.c_size_t(0)
    _check(lib().gsi_stack_workspace_size(arr, len(maps), T, ctypes.byref(n)))
    return n.value


def new_workspace(nbytes: int, device="cuda", stream=None) -> torch.Tensor:
    """A zero-initialised workspace of at least nbytes (256-byte aligned)."""
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    _check(lib().gsi_workspace_init(_ptr(ws), ws.numel(), _stream(stream)))
    return ws


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    code = ctypes.c_uint32(0)
    st = lib().gsi_workspace_status(_ptr(ws), ctypes.byref(code), _stream(stream))
    if st not in (0, 5):
        _check(st)
    return code.value


def linear(m: Map, X: torch.Tensor, eps: float, Y=None, flags=None, rho=None, workspace=None,
           path: str = "auto", want_rho: bool = True, stream=None):
    """The gated linear map over the T tokens of X; returns (Y, flags, rho)."""
    _require_cuda(X)
    T = X.shape[0]
    dev = X.device
    if Y is None:
        Y = torch.empty(T, m.d_out, dtype=torch.float32, device=dev)
    if flags is None:
        flags = torch.empty(T, dtype=torch.uint8, device=dev)
    if rho is None and want_rho:
        rho = torch.empty(T, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = new_workspace(workspace_size(m, T, path), dev, stream)
    desc = m.desc()
    _check(lib().gsi_linear_ex(ctypes.byref(desc), _ptr(X), T, float(eps), _ptr(Y), _ptr(flags),
                               _ptr(rho), _ptr(workspace), workspace.numel(), PATHS[path],
                               _stream(stream)))
    return Y, flags, rho


def path_errors(m: Map, X: torch.Tensor, workspace=None, stream=None):
    """Both candidate outputs of every token and their distance.

    Returns (Y_fast, Y_slow, rho, err, ynorm): M g_t and W x_t rows, the
    residual ratios, ||Y_fast[t] - Y_slow[t]|| and ||Y_slow[t]||.
    """
    _require_cuda(X)
    T, dev = X.shape[0], X.device
    f32 = dict(dtype=torch.float32, device=dev)
    Yf, Ys = torch.empty(T, m.d_out, **f32), torch.empty(T, m.d_out, **f32)
    rho, err, ynorm = torch.empty(T, **f32), torch.empty(T, **f32), torch.empty(T, **f32)
    flags = torch.empty(T, dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = new_workspace(workspace_size(m, T), dev, stream)
    desc = m.desc()
    _check(lib().gsi_path_errors(ctypes.byref(desc), _ptr(X), T, _ptr(Yf), _ptr(Ys), _ptr(flags), _ptr(rho),
                                 _ptr(err), _ptr(ynorm), _ptr(workspace), workspace.numel(), _stream(stream)))
    return Yf, Ys, rho, err, ynorm


def eps_sweep(rho: torch.Tensor, err: torch.Tensor, ynorm: torch.Tensor, eps, tokens_per_call: int = 1,
              stream=None):
    """The gate at each threshold of `eps`; returns (n_slow, n_slow_calls, rel_err) device tensors."""
    _require_cuda(rho, err, ynorm)
    dev = rho.device
    e = torch.as_tensor(list(eps), dtype=torch.float32).to(dev)
    n = e.numel()
    n_slow = torch.empty(n, dtype=torch.int32, device=dev)
    n_calls = torch.empty(n, dtype=torch.int32, device=dev)
    rel = torch.empty(n, dtype=torch.float32, device=dev)
    _check(lib().gsi_eps_sweep(_ptr(rho), _ptr(err), _ptr(ynorm), rho.numel(), _ptr(e), n, int(tokens_per_call),
                               _ptr(n_slow), _ptr(n_calls), _ptr(rel), _stream(stream)))
    return n_slow, n_calls, rel


def basis_orthonormalize(Vt: torch.Tensor, stream=None):
    """DGKS Gram-Schmidt of the rows of Vt (k x d float32) in place; returns
    (Vt, n_reorth) with n_reorth a device int32 tensor."""
    _require_cuda(Vt)
    n = torch.zeros(1, dtype=torch.int32, device=Vt.device)
    _check(lib().gsi_basis_orthonormalize(_ptr(Vt), Vt.shape[0], Vt.shape[1], _ptr(n), _stream(stream)))
    return Vt, n


def basis_step(X: torch.Tensor, Vt: torch.Tensor, work=None, stream=None):
    """One correction step Vt <- DGKS((X^T X V)^T) on the calibration block X
    (T x d, float32 or bfloat16); returns (Vt, n_reorth)."""
    _require_cuda(X, Vt)
    T, d = X.shape
    k = Vt.shape[0]
    if work is None:
        work = new_workspace(int(lib().gsi_basis_step_work_bytes(T, d, k)), X.device, stream)
    n = torch.zeros(1, dtype=torch.int32, device=X.device)
    _check(lib().gsi_basis_step(_ptr(X), _dtype_code(X.dtype), T, d, k, _ptr(Vt), _ptr(work), work.numel(),
                                _ptr(n), _stream(stream)))
    return Vt, n


def basis_coherence(Vt_a: torch.Tensor, Vt_b: torch.Tensor, stream=None) -> torch.Tensor:
    """||Va^T Vb||_F^2 / k for two orthonormal bases held as k x d rows."""
    _require_cuda(Vt_a, Vt_b)
    k, d = Vt_a.shape
    out = torch.empty(1, dtype=torch.float32, device=Vt_a.device)
    work = torch.empty(k * k, dtype=torch.float32, device=Vt_a.device)
    _check(lib().gsi_basis_coherence(_ptr(Vt_a), _ptr(Vt_b), k, d, _ptr(out), _ptr(work), _stream(stream)))
    return out


def basis_export(Vt: torch.Tensor, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The basis in a map's layout: V = Vt^T (d x k, row-major) in `dtype`."""
    _require_cuda(Vt)
    k, d = Vt.shape
    V = torch.empty(d, k, dtype=dtype, device=Vt.device)
    _check(lib().gsi_basis_export(_ptr(Vt), k, d, _ptr(V), _dtype_code(dtype), _stream(stream)))
    return V


def gate(m: Map, X: torch.Tensor, eps: float, workspace=None, G=None, rho=None, flags=None,
         stream=None):
    """Projections, residual ratios and flags only; returns (G, rho, flags)."""
    _require_cuda(X)
    T = X.shape[0]
    if G is None:
        G = torch.empty(T, m.k, dtype=torch.float32, device=X.device)
    if rho is None:
        rho = torch.empty(T, dtype=torch.float32, device=X.device)
    if flags is None:
        flags = torch.empty(T, dtype=torch.uint8, device=X.device)
    if workspace is None:
        workspace = new_workspace(workspace_size(m, T, "stream"), X.device, stream)
    desc = m.desc()
    _check(lib().gsi_gate(ctypes.byref(desc), _ptr(X), T, float(eps), _ptr(G), _ptr(rho),
                          _ptr(flags), _ptr(workspace), workspace.numel(), _stream(stream)))
    return G, rho, flags


def residual_check(m: Map, X: torch.Tensor, G: torch.Tensor, rho: torch.Tensor, work=None, stream=None):
    """The gate's residual ratios checked against the explicit residual
    x - V g (a second pass over V); returns (rho_explicit, max_dev) with
    max_dev = max_t |rho_t^2 - rho_explicit_t^2| (device tensors)."""
    _require_cuda(X, G, rho)
    T = X.shape[0]
    rho_x = torch.empty(T, dtype=torch.float32, device=X.device)
    dev = torch.empty(1, dtype=torch.float32, device=X.device)
    if work is None:
        work = torch.empty(max(int(lib().gsi_residual_check_work_bytes(m.d, T)), 256), dtype=torch.uint8,
                           device=X.device)
    desc = m.desc()
    _check(lib().gsi_residual_check(ctypes.byref(desc), _ptr(X), T, _ptr(G), _ptr(rho), _ptr(rho_x), _ptr(dev),
                                    _ptr(work), work.numel(), _stream(stream)))
    return rho_x, dev


def apply(m: Map, X: torch.Tensor, G: torch.Tensor, workspace: torch.Tensor, Y=None, stream=None):
    """Fast / slow paths for the tokens of the preceding gate() on `workspace`."""
    _require_cuda(X, G)
    T = X.shape[0]
    if Y is None:
        Y = torch.empty(T, m.d_out, dtype=torch.float32, device=X.device)
    desc = m.desc()
    _check(lib().gsi_apply(ctypes.byref(desc), _ptr(X), _ptr(G), T, _ptr(Y), _ptr(workspace),
                           workspace.numel(), _stream(stream)))
    return Y


def compact(flags: torch.Tensor, stream=None):
    """Stable fast / slow index lists: returns (idx (2T int32), counts (2 int32))."""
    _require_cuda(flags)
    T = flags.shape[0]
    idx = torch.full((2 * max(T, 1),), -1, dtype=torch.int32, device=flags.device)
    counts = torch.zeros(2, dtype=torch.int32, device=flags.device)
    _check(lib().gsi_compact(_ptr(flags), T, _ptr(idx), _ptr(counts), _stream(stream)))
    return idx, counts


STACK_MODES = {"auto": 0, "per_map": 1, "persistent": 2}


def stack(maps, Xs, eps: float, Ys=None, flags=None, workspace=None, stream=None, mode: str = "auto"):
    """The gated map over a list of maps, each with its own tokens."""
    n = len(maps)
    T = Xs[0].shape[0]
    dev = Xs[0].device
    if Ys is None:
        Ys = [torch.empty(T, m.d_out, dtype=torch.float32, device=dev) for m in maps]
    if flags is None:
        flags = [torch.empty(T, dtype=torch.uint8, device=dev) for _ in maps]
    if workspace is None:
        workspace = new_workspace(stack_workspace_size(maps, T), dev, stream)
    args = stack_args(maps, Xs, Ys, flags)
    _check(lib().gsi_stack_ex(args[0], n, args[1], T, float(eps), args[2], args[3],
                              _ptr(workspace), workspace.numel(), STACK_MODES[mode], _stream(stream)))
    return Ys, flags


def stack_args(maps, Xs, Ys, flags):
    """ctypes arrays for gsi_stack (build once, reuse across calls)."""
    n = len(maps)
    vp = ctypes.c_void_p
    return ((MapDesc * n)(*[m.desc() for m in maps]),
            (vp * n)(*[x.data_ptr() for x in Xs]),
            (vp * n)(*[y.data_ptr() for y in Ys]),
            (vp * n)(*[f.data_ptr() for f in flags]))


def stack_raw(args, n, T, eps, workspace, stream=None, mode: str = "auto"):
    """gsi_stack_ex on prepared ctypes arrays (no per-call Python allocation)."""
    _check(lib().gsi_stack_ex(args[0], n, args[1], T, float(eps), args[2], args[3],
                              _ptr(workspace), workspace.numel(), STACK_MODES[mode], _stream(stream)))


# ---------------------------------------------------------------- serving operators
# What stands between the gated maps of a decoder layer: pages and slots of a
# step's tokens, the paged key/value cache, attention over it, and the norms
# with gate and residual.  Outputs and workspaces may be passed in (a serving
# loop keeps them); what is not passed is allocated by PyTorch on `stream`.
# All tensors of a call lie on the current CUDA device.

PLAN_BAD_LENGTH, PLAN_TABLE_FULL, PLAN_NO_PAGES, PLAN_TOO_MANY_TOKENS = 1, 2, 4, 8
NORMS = {"none": 0, "rms": 1, "layer": 2}


def _on_stream(stream):
    """Allocations inside belong to the stream that uses them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


# (The calls below take microseconds on the GPU: their checks are written for
# the time they take here.)
_I32, _I64 = torch.int32, torch.int64
_DTYPES = {torch.float32: GSI_F32, torch.bfloat16: GSI_BF16}


def _device(name, t) -> int:
    """The device of a call's tensors: kernels run on the current one, and only there are its pointers good."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be a tensor of the current CUDA device, not of {t.device}")
    return dev


def _ints(name, t, n, dev, dtype=_I32):
    """A contiguous integer tensor of n elements on this device."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous tensor of {n} {dtype} on cuda:{dev}, "
                         f"not {tuple(t.shape)} {t.dtype} on {t.device}")


def _like(name, t, shape, dtype, dev):
    """A contiguous tensor of this shape and type on this device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {tuple(shape)} {dtype} on cuda:{dev}, "
                         f"not {tuple(t.shape)} {t.dtype} on {t.device}")


def _float_code(t) -> int:
    code = _DTYPES.get(t.dtype)
    return _dtype_code(t.dtype) if code is None else code


@dataclass
class PagedCache:
    """Keys and values in pages: two (pages, heads, page_size, head_dim) tensors
    of one dtype (float32 or bfloat16) and one layout.  Only head_dim has to be
    contiguous: a (pages, page_size, heads, head_dim) buffer is passed as its
    permuted view."""
    K: torch.Tensor
    V: torch.Tensor

    @classmethod
    def empty(cls, n_pages: int, n_heads: int, page_size: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        return cls(*(torch.empty(n_pages, n_heads, page_size, head_dim, dtype=dtype, device=device) for _ in range(2)))

    def desc(self) -> CacheDesc:
        K, V = self.K, self.V
        shape, st = K.shape, K.stride()
        if len(shape) != 4 or V.shape != shape or V.stride() != st or V.dtype is not K.dtype:
            raise ValueError("K and V must be two (pages, heads, page_size, head_dim) tensors of one dtype and layout")
        if not K.is_cuda or V.get_device() != K.get_device() or st[3] != 1:
            raise ValueError("K and V must be tensors of one CUDA device with contiguous head_dim")
        n, h, p, d = shape
        return CacheDesc(n, p, h, d, _float_code(K), st[0], st[1], st[2], K.data_ptr(), V.data_ptr())


@dataclass
class PagedPlan:
    """One step's plan (device tensors): q_start (requests + 1), kv_len (requests),
    slots (int64), token_req and positions (one a token), n_free and status (1)."""
    q_start: torch.Tensor
    kv_len: torch.Tensor
    slots: torch.Tensor
    token_req: torch.Tensor
    positions: torch.Tensor
    n_free: torch.Tensor
    status: torch.Tensor

    @classmethod
    def empty(cls, n_requests: int, n_tokens: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(n_requests + 1, **i32), torch.empty(n_requests, **i32),
                   torch.empty(n_tokens, dtype=torch.int64, device=device), torch.empty(n_tokens, **i32),
                   torch.empty(n_tokens, **i32), torch.empty(1, **i32), torch.empty(1, **i32))


def paged_plan(cached: torch.Tensor, fresh: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
               n_free: torch.Tensor, page_size: int, n_tokens: int = None, plan: PagedPlan = None,
               stream=None) -> PagedPlan:
    """Pages and slots of a step in which request r, with cached[r] tokens in the
    pages of table[r], appends fresh[r] tokens (int32 tensors).  The pages come
    off the end of free_pages[:n_free]; the table's new entries are written in
    place.  n_tokens: the capacity of the token arrays (the new tokens' number,
    or more, the rest padded with -1).  plan.status is 0, or PLAN_ bits and
    nothing planned; it stays on the device (check it where the step's tokens
    are read back)."""
    R = cached.numel()
    if plan is None:
        if n_tokens is None:
            raise ValueError("n_tokens or a plan to write is needed")
        with _on_stream(stream):
            plan = PagedPlan.empty(R, n_tokens, cached.device)
    N = plan.slots.numel()
    if n_tokens is not None and n_tokens != N:
        raise ValueError(f"plan holds {N} tokens, not {n_tokens}")
    if table.dim() != 2 or table.shape[0] != R:
        raise ValueError(f"table must be ({R}, pages), not {tuple(table.shape)}")
    width = table.shape[1]
    capacity = free_pages.numel()
    q_start, kv_len, slots, req, pos, left, status = (plan.q_start, plan.kv_len, plan.slots, plan.token_req, plan.positions,
                                                      plan.n_free, plan.status)
    dev = _device("cached", cached)
    _ints("cached", cached, R, dev)
    _ints("fresh", fresh, R, dev)
    _ints("table", table, R * width, dev)
    _ints("free_pages", free_pages, capacity, dev)
    _ints("n_free", n_free, 1, dev)
    _ints("plan.q_start", q_start, R + 1, dev)
    _ints("plan.kv_len", kv_len, R, dev)
    _ints("plan.slots", slots, N, dev, _I64)
    _ints("plan.token_req", req, N, dev)
    _ints("plan.positions", pos, N, dev)
    _ints("plan.n_free", left, 1, dev)
    _ints("plan.status", status, 1, dev)
    _check(lib().gsi_paged_plan(cached.data_ptr(), fresh.data_ptr(), R, table.data_ptr(), width, free_pages.data_ptr(),
                                capacity, n_free.data_ptr(), page_size, N, q_start.data_ptr(), kv_len.data_ptr(),
                                slots.data_ptr(), req.data_ptr(), pos.data_ptr(), left.data_ptr(), status.data_ptr(),
                                _raw_stream(stream, cached)))
    return plan


def cache_append(cache: PagedCache, rows: torch.Tensor, slots: torch.Tensor, n_q_heads: int, Q=None, stream=None):
    """The rows of a qkv map (T x (n_q_heads + 2 heads) head_dim, float32 or
    bfloat16, rows contiguous): keys and values into the cache at `slots`
    (negative: padding), queries to Q (T, n_q_heads, head_dim), returned."""
    c = cache.desc()
    dev = _device("the cache", cache.K)
    T = slots.numel()
    D = c.head_dim
    st = rows.stride()
    if rows.shape != (T, (n_q_heads + 2 * c.n_heads) * D) or rows.get_device() != dev or (st[1] != 1 and T):
        raise ValueError(f"rows must be rows of ({T}, {(n_q_heads + 2 * c.n_heads) * D}) on the cache's device, "
                         f"not {tuple(rows.shape)} on {rows.device}")
    _ints("slots", slots, T, dev, _I64)
    if Q is None:
        with _on_stream(stream):
            Q = torch.empty(T, n_q_heads, D, dtype=cache.K.dtype, device=rows.device)
    else:
        _like("Q", Q, (T, n_q_heads, D), cache.K.dtype, dev)
    _check(lib().gsi_cache_append(c, rows.data_ptr(), _float_code(rows), st[0], slots.data_ptr(), T, n_q_heads,
                                  Q.data_ptr(), _raw_stream(stream, rows)))
    return Q


def paged_attention_workspace_size(cache: PagedCache, n_q_heads: int) -> int:
    c = cache.desc()
    n = int(lib().gsi_paged_attention_workspace_size(ctypes.byref(c), n_q_heads))
    if n == 0:
        raise GsiError(1, lib().gsi_last_error().decode() or "no attention of this shape")
    return n


def paged_attention(cache: PagedCache, Q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
                    table: torch.Tensor, max_q: int = None, scale: float = None, causal: bool = True, window: int = 0,
                    out=None, workspace=None, stream=None, lse=None):
    """Attention of every request's new tokens Q (N, heads, head_dim; rows of the
    cache's dtype, any stride between tokens) over its cached keys, as planned
    by paged_plan; returns out (N, heads, head_dim).  causal: the new tokens are
    the last ones of the request's kv_len keys; window > 0: a token sees only
    that many keys, its own the last.  causal=False: every key (cross attention
    to cached states).  A row that sees no key gives zeros (one whose scores are
    all -inf NaN); rows of no request are not written.  max_q: a bound on a
    request's new tokens, for the choice of kernel (a wrong one costs time, not
    results).  scale defaults to head_dim ** -0.5.  Without a workspace every
    call allocates and zeroes one (some 40 MB at 128 columns): a serving loop
    keeps one, of paged_attention_workspace_size bytes from new_workspace.
    lse: float32 (N, heads) to write the logarithm of each row's sum of weights
    to, for key_weights."""
    c = cache.desc()
    dev = _device("the cache", cache.K)
    shape, st = Q.shape, Q.stride()
    if len(shape) != 3 or Q.get_device() != dev or Q.dtype is not cache.K.dtype or shape[2] != c.head_dim:
        raise ValueError(f"Q must be a (tokens, heads, {c.head_dim}) tensor of {cache.K.dtype} on cuda:{dev}, "
                         f"not {tuple(shape)} {Q.dtype} on {Q.device}")
    N, H, D = shape
    if N and (st[2] != 1 or (H > 1 and st[1] != D)):
        raise ValueError("the heads of a token of Q must be contiguous")
    R = kv_len.numel()
    if table.dim() != 2 or table.shape[0] != R:
        raise ValueError(f"table must be ({R}, pages), not {tuple(table.shape)}")
    width = table.shape[1]
    _ints("table", table, R * width, dev)
    _ints("q_start", q_start, R + 1, dev)
    _ints("kv_len", kv_len, R, dev)
    if out is None:
        with _on_stream(stream):
            out = torch.empty(N, H, D, dtype=Q.dtype, device=Q.device)
    else:
        _like("out", out, shape, Q.dtype, dev)
    if workspace is None:
        with _on_stream(stream):
            workspace = new_workspace(paged_attention_workspace_size(cache, H), Q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}, not on {workspace.device}")
    if lse is not None:
        _like("lse", lse, (N, H), torch.float32, dev)
    _check(lib().gsi_paged_attention_lse(c, Q.data_ptr(), st[0], N, H, q_start.data_ptr(), kv_len.data_ptr(),
                                         table.data_ptr(), width, R, N if max_q is None else max_q,
                                         D ** -0.5 if scale is None else scale, 1 if causal else 0, window, out.data_ptr(),
                                         None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                         _raw_stream(stream, Q)))
    return out


@dataclass
class Norm:
    """A norm over a row: kind "rms", "layer" or "none", float32 weight and bias (or None)."""
    kind: str
    weight: torch.Tensor = None
    bias: torch.Tensor = None
    eps: float = 1e-5

    def desc(self, d: int, dev: int = None) -> NormDesc:
        w, b = self.weight, self.bias
        if w is not None:
            _like("norm weight", w, (d,), torch.float32, max(w.get_device(), 0) if dev is None else dev)
        if b is not None:
            _like("norm bias", b, (d,), torch.float32, max(b.get_device(), 0) if dev is None else dev)
        return NormDesc(NORMS[self.kind], self.eps, None if w is None else w.data_ptr(),
                        None if b is None else b.data_ptr())


def norm_residual(h: torch.Tensor, y: torch.Tensor = None, post: Norm = None, pre: Norm = None, gate=None,
                  gate_index=None, alpha: float = 1.0, h_out=None, x=None, x_dtype=torch.bfloat16, stream=None):
    """The end of one block and the beginning of the next, in one pass over T x d
    rows: h_out = alpha h + gate post(y), x = pre(h_out); returns (h_out, x).
    h, y, x: float32 or bfloat16.  gate: float32, (d,) for every token or
    (n, d) with gate_index (T int32) naming each token's row (a plan's
    token_req, for a gate per request).  h_out may be h."""
    shape = h.shape
    T, d = shape
    dev = _device("h", h)
    if not h.is_contiguous():
        raise ValueError("h must be contiguous")
    if y is not None:
        _like("y", y, shape, y.dtype, dev)
    rows = 0
    if gate is not None:
        rows = gate.numel() // d
        _like("gate", gate, gate.shape[:-1] + (d,), torch.float32, dev)
        if gate_index is not None:
            _ints("gate_index", gate_index, T, dev)
        elif rows != 1:
            raise ValueError("a gate of several rows needs gate_index")
        if rows == 0 and T:
            raise ValueError("a gate needs a row")
    if h_out is None:
        with _on_stream(stream):
            h_out = torch.empty_like(h)
    else:
        _like("h_out", h_out, shape, h.dtype, dev)
    if x is None:
        with _on_stream(stream):
            x = torch.empty(T, d, dtype=x_dtype, device=h.device)
    else:
        _like("x", x, shape, x.dtype, dev)
    _check(lib().gsi_norm_residual(h.data_ptr(), _float_code(h), None if y is None else y.data_ptr(),
                                   0 if y is None else _float_code(y), T, d, alpha,
                                   None if post is None else post.desc(d, dev), None if gate is None else gate.data_ptr(), rows,
                                   None if gate_index is None else gate_index.data_ptr(),
                                   None if pre is None else pre.desc(d, dev), h_out.data_ptr(), x.data_ptr(), _float_code(x),
                                   _raw_stream(stream, h)))
    return h_out, x


ROTARY_LAYOUTS = {"half": 0, "pairs": 1}
ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


@dataclass
class Rotary:
    """The positions' angles: the first dim values of a head are turned, pair i
    being values i and dim / 2 + i (layout "half") or 2 i and 2 i + 1 ("pairs"),
    by position * w_i, and multiplied by scale.  phases: the w_i in units of
    2^-64 of a turn, int64 (dim / 2) on the device."""
    dim: int
    phases: torch.Tensor
    layout: str = "half"
    scale: float = 1.0

    @classmethod
    def from_rates(cls, rates, layout: str = "half", scale: float = 1.0, device="cuda"):
        """From the w_i in radians a position (numbers of up to 2^40, kept in 64 bits)."""
        n = len(rates)
        w, out = (ctypes.c_double * n)(*[float(r) for r in rates]), (ctypes.c_uint64 * n)()
        _check(lib().gsi_rotary_phases(w, n, out))
        phases = torch.tensor([p - 2 ** 64 if p >= 2 ** 63 else p for p in out], dtype=torch.int64, device=device)
        return cls(2 * n, phases, layout, scale)

    @classmethod
    def make(cls, dim: int, base: float = 10000.0, layout: str = "half", scaling: str = "none", factor: float = 1.0,
             context: float = 0.0, fast: float = 0.0, slow: float = 0.0, device="cuda"):
        """w_i = base ** (-2 i / dim), scaled for contexts longer than `context` (include/gsi.h has the forms):
        "linear", "ntk", "yarn" (fast, slow: turns within the context; 32 and 1 by default) or "bands" (4 and 1)."""
        rates, scale = cls.rates(dim, base, scaling, factor, context, fast, slow)
        return cls.from_rates(rates, layout, scale, device)

    @staticmethod
    def rates(dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, context: float = 0.0,
              fast: float = 0.0, slow: float = 0.0):
        """The w_i (radians a position) and the scale of `make`."""
        default = {"yarn": (32.0, 1.0), "bands": (4.0, 1.0)}.get(scaling, (0.0, 0.0))
        out, scale = (ctypes.c_double * max(dim // 2, 1))(), ctypes.c_float()
        _check(lib().gsi_rotary_rates(dim, base, ROTARY_SCALINGS[scaling], factor, context, fast or default[0],
                                      slow or default[1], out, ctypes.byref(scale)))
        return list(out), scale.value

    def desc(self, dev: int) -> RotaryDesc:
        _ints("rotary.phases", self.phases, self.dim // 2, dev, _I64)
        return RotaryDesc(self.dim, ROTARY_LAYOUTS[self.layout], self.scale, self.phases.data_ptr())


def rotary_append(cache: PagedCache, rows: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor, n_q_heads: int,
                  rotary: Rotary, token_req=None, offsets=None, Q=None, stream=None):
    """cache_append with queries and keys turned by their positions (int32, one a
    token), plus offsets[token_req] where a request's places have moved
    (cache_evict's offsets_out and a plan's token_req)."""
    c = cache.desc()
    dev = _device("the cache", cache.K)
    T = slots.numel()
    D = c.head_dim
    st = rows.stride()
    if rows.shape != (T, (n_q_heads + 2 * c.n_heads) * D) or rows.get_device() != dev or (st[1] != 1 and T):
        raise ValueError(f"rows must be rows of ({T}, {(n_q_heads + 2 * c.n_heads) * D}) on the cache's device, "
                         f"not {tuple(rows.shape)} on {rows.device}")
    _ints("slots", slots, T, dev, _I64)
    _ints("positions", positions, T, dev)
    R = 0
    if offsets is not None:
        R = offsets.numel()
        _ints("offsets", offsets, R, dev)
        if token_req is not None:
            _ints("token_req", token_req, T, dev)
        elif R != 1:
            raise ValueError("offsets of several requests need token_req")
    if Q is None:
        with _on_stream(stream):
            Q = torch.empty(T, n_q_heads, D, dtype=cache.K.dtype, device=rows.device)
    else:
        _like("Q", Q, (T, n_q_heads, D), cache.K.dtype, dev)
    _check(lib().gsi_rotary_append(c, rows.data_ptr(), _float_code(rows), st[0], slots.data_ptr(), positions.data_ptr(),
                                   None if token_req is None else token_req.data_ptr(),
                                   None if offsets is None else offsets.data_ptr(), R, T, n_q_heads, rotary.desc(dev),
                                   Q.data_ptr(), _raw_stream(stream, rows)))
    return Q


@dataclass
class KeyMarks:
    """What eviction goes by: for every page, head and token of a cache the
    attention weight that the key has gathered (float32) and its position in
    the sequence (int32), two dense (pages, heads, page_size) tensors."""
    weight: torch.Tensor
    place: torch.Tensor

    @classmethod
    def empty(cls, cache: PagedCache):
        """Marks of a cache's shape (what they hold means nothing until key_weights has written it)."""
        shape, dev = cache.K.shape[:3], cache.K.device
        return cls(torch.empty(shape, dtype=torch.float32, device=dev), torch.empty(shape, dtype=torch.int32, device=dev))

    def desc(self, cache: PagedCache, dev: int) -> MarksDesc:
        _like("marks.weight", self.weight, cache.K.shape[:3], torch.float32, dev)
        _like("marks.place", self.place, cache.K.shape[:3], _I32, dev)
        return MarksDesc(self.weight.data_ptr(), self.place.data_ptr())


def key_weights_workspace_size() -> int:
    return int(lib().gsi_key_weights_workspace_size())


def key_weights(cache: PagedCache, Q: torch.Tensor, lse: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
                table: torch.Tensor, marks: KeyMarks, held=None, offsets=None, max_q: int = None, scale: float = None,
                causal: bool = True, workspace=None, stream=None) -> KeyMarks:
    """The attention weight that every key receives from the tokens Q, whose
    attention left lse (paged_attention's, the same Q, q_start, kv_len, table,
    scale and causal): added to the marks of the first held[r] keys of request r
    (a plan's cached lengths), the beginning of the others', which get the
    position place + offsets[r] (cache_evict's offsets_out).  held None: no key
    has marks yet.  Q may be the last tokens only of those that came in.  No page
    may belong to two requests (a shared beginning): their sums would overwrite
    each other."""
    c = cache.desc()
    dev = _device("the cache", cache.K)
    shape, st = Q.shape, Q.stride()
    if len(shape) != 3 or Q.get_device() != dev or Q.dtype is not cache.K.dtype or shape[2] != c.head_dim:
        raise ValueError(f"Q must be a (tokens, heads, {c.head_dim}) tensor of {cache.K.dtype} on cuda:{dev}, "
                         f"not {tuple(shape)} {Q.dtype} on {Q.device}")
    N, H, D = shape
    if N and (st[2] != 1 or (H > 1 and st[1] != D)):
        raise ValueError("the heads of a token of Q must be contiguous")
    R = kv_len.numel()
    if table.dim() != 2 or table.shape[0] != R:
        raise ValueError(f"table must be ({R}, pages), not {tuple(table.shape)}")
    width = table.shape[1]
    _like("lse", lse, (N, H), torch.float32, dev)
    _ints("table", table, R * width, dev)
    _ints("q_start", q_start, R + 1, dev)
    _ints("kv_len", kv_len, R, dev)
    if held is not None:
        _ints("held", held, R, dev)
    if offsets is not None:
        _ints("offsets", offsets, R, dev)
    m = marks.desc(cache, dev)
    if workspace is None:
        with _on_stream(stream):
            workspace = new_workspace(key_weights_workspace_size(), Q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}, not on {workspace.device}")
    _check(lib().gsi_key_weights(c, Q.data_ptr(), st[0], N, H, lse.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                                 None if held is None else held.data_ptr(), None if offsets is None else offsets.data_ptr(),
                                 table.data_ptr(), width, R, N if max_q is None else max_q,
                                 D ** -0.5 if scale is None else scale, 1 if causal else 0, m, workspace.data_ptr(),
                                 workspace.numel(), _raw_stream(stream, Q)))
    return marks


def cache_evict_workspace_size(cache: PagedCache, n_requests: int, budget: int) -> int:
    c = cache.desc()
    n = int(lib().gsi_cache_evict_workspace_size(ctypes.byref(c), n_requests, budget))
    if n == 0:
        raise GsiError(1, lib().gsi_last_error().decode() or "no eviction of this shape")
    return n


def cache_evict(cache: PagedCache, kv_len: torch.Tensor, table: torch.Tensor, marks: KeyMarks, budget: int,
                recent: int = 0, sinks: int = 0, offsets=None, kept=None, offsets_out=None, workspace=None, stream=None):
    """Every request of more than `budget` keys keeps that many, for each head by
    itself: those of the last `recent` positions, of the first `sinks`, and those
    that gathered the most weight; the kept ones close the gaps (their order
    changes).  Returns (kept, offsets_out): the lengths then, and offsets plus
    the keys given up (the offsets of the next rotary_append, key_weights and
    cache_evict).  paged_trim returns the pages: once for layers that share the
    table.  No page may belong to two requests."""
    c = cache.desc()
    dev = _device("the cache", cache.K)
    R = kv_len.numel()
    if table.dim() != 2 or table.shape[0] != R:
        raise ValueError(f"table must be ({R}, pages), not {tuple(table.shape)}")
    width = table.shape[1]
    _ints("table", table, R * width, dev)
    _ints("kv_len", kv_len, R, dev)
    if offsets is not None:
        _ints("offsets", offsets, R, dev)
    m = marks.desc(cache, dev)
    if kept is None or offsets_out is None or workspace is None:
        with _on_stream(stream):
            kept = torch.empty_like(kv_len) if kept is None else kept
            offsets_out = torch.empty_like(kv_len) if offsets_out is None else offsets_out
            if workspace is None:
                workspace = new_workspace(cache_evict_workspace_size(cache, R, budget), kv_len.device, stream)
    _ints("kept", kept, R, dev)
    _ints("offsets_out", offsets_out, R, dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}, not on {workspace.device}")
    _check(lib().gsi_cache_evict(c, kv_len.data_ptr(), table.data_ptr(), width, R, m, budget, recent, sinks,
                                 None if offsets is None else offsets.data_ptr(), kept.data_ptr(), offsets_out.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(), _raw_stream(stream, kv_len)))
    return kept, offsets_out


@dataclass
class Verdict:
    """Of one step's drafts (device tensors): out (one a row: a request's next
    tokens, then -1), accepted (requests) and kept (the requests' lengths, or None)."""
    out: torch.Tensor
    accepted: torch.Tensor
    kept: torch.Tensor = None


def verify_drafts(target: torch.Tensor, draft, tokens: torch.Tensor, uniforms: torch.Tensor, samples: torch.Tensor,
                  q_start: torch.Tensor, kv_len=None, out=None, accepted=None, kept=None, stream=None) -> Verdict:
    """Drafted tokens against the target's probabilities (N, vocab), row
    q_start[r] being request r's last token and the rows behind it its drafts
    (tokens, int32): row t's draft tokens[t + 1] stands if uniforms[t] draft <
    target; the first that does not is replaced by a sample of what the draft
    leaves of the target, behind drafts that all stand comes one of the target
    (samples: a number within [0, 1) a request).  draft: (N, vocab)
    probabilities, or None for drafts that are certain.  kv_len gives kept, the
    lengths without the places of drafts that do not stand (for paged_trim)."""
    dev = _device("target", target)
    if target.dim() != 2 or (draft is not None and (draft.shape != target.shape or draft.get_device() != dev)):
        raise ValueError("target and draft must be (tokens, vocabulary) tensors of one shape and device")
    N, V = target.shape
    ts, ds = target.stride(), (0, 1) if draft is None else draft.stride()
    if N and V > 1 and (ts[1] != 1 or ds[1] != 1):
        raise ValueError("the rows of target and draft must be contiguous")
    R = q_start.numel() - 1
    if R < 0:
        raise ValueError("q_start must have one number more than there are requests")
    _ints("tokens", tokens, N, dev)
    _like("uniforms", uniforms, (N,), torch.float32, dev)
    _like("samples", samples, (R,), torch.float32, dev)
    _ints("q_start", q_start, R + 1, dev)
    if kv_len is not None:
        _ints("kv_len", kv_len, R, dev)
    elif kept is not None:
        raise ValueError("kept needs kv_len")
    if out is None or accepted is None or (kept is None and kv_len is not None):
        with _on_stream(stream):
            out = torch.empty(N, dtype=_I32, device=target.device) if out is None else out
            accepted = torch.empty(R, dtype=_I32, device=target.device) if accepted is None else accepted
            if kept is None and kv_len is not None:
                kept = torch.empty(R, dtype=_I32, device=target.device)
    _ints("out", out, N, dev)
    _ints("accepted", accepted, R, dev)
    if kept is not None:
        _ints("kept", kept, R, dev)
    _check(lib().gsi_verify_drafts(target.data_ptr(), _float_code(target), ts[0], None if draft is None else draft.data_ptr(),
                                   0 if draft is None else _float_code(draft), ds[0], N, V, tokens.data_ptr(),
                                   uniforms.data_ptr(), samples.data_ptr(), q_start.data_ptr(),
                                   None if kv_len is None else kv_len.data_ptr(), R, out.data_ptr(), accepted.data_ptr(),
                                   None if kept is None else kept.data_ptr(), _raw_stream(stream, target)))
    return Verdict(out, accepted, kept)


def paged_trim(kv_len: torch.Tensor, kept: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
               n_free: torch.Tensor, page_size: int, n_free_out=None, status=None, stream=None):
    """The pages that requests of kv_len tokens no longer fill when they keep
    kept[r] of them (0: the request is done), back on free_pages[n_free:]; a plan
    that needs as many takes them in the same order again.  Returns (n_free_out,
    status): the free pages then, and 0 or PLAN_ bits and nothing given back."""
    dev = _device("kv_len", kv_len)
    R, capacity = kv_len.numel(), free_pages.numel()
    if table.dim() != 2 or table.shape[0] != R:
        raise ValueError(f"table must be ({R}, pages), not {tuple(table.shape)}")
    width = table.shape[1]
    _ints("kv_len", kv_len, R, dev)
    _ints("kept", kept, R, dev)
    _ints("table", table, R * width, dev)
    _ints("free_pages", free_pages, capacity, dev)
    _ints("n_free", n_free, 1, dev)
    if n_free_out is None or status is None:
        with _on_stream(stream):
            n_free_out = torch.empty_like(n_free) if n_free_out is None else n_free_out
            status = torch.empty_like(n_free) if status is None else status
    _ints("n_free_out", n_free_out, 1, dev)
    _ints("status", status, 1, dev)
    _check(lib().gsi_paged_trim(kv_len.data_ptr(), kept.data_ptr(), R, table.data_ptr(), width, free_pages.data_ptr(),
                                capacity, n_free.data_ptr(), page_size, n_free_out.data_ptr(), status.data_ptr(),
                                _raw_stream(stream, kv_len)))
    return n_free_out, status
