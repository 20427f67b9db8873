// The end of one block and the beginning of the next in one pass:
//   h' = alpha h + gate * post(y),   x = pre(h').

#include <type_traits>

#include "gsi_common.cuh"
#include "gsi_kernels.h"

namespace gsi {

// Every value of a row stays in registers from its load to its stores: y and h
// are read once, h' and x written once, and the norms' sums are block
// reductions between (LAYER: the mean first, then the centred squares, so no
// difference of large sums appears).  A thread holds pieces of four values, the
// next thread the next piece: a warp's 16-byte accesses cover whole lines (with
// eight float32 values a thread every access touched half of twice the sectors).
//
// Few tokens are latency: a CTA a token (one of 4096: 2.5 us).  Many are bytes, and a CTA a token
// waits for its first loads and its weights most of its life: there the CTAs
// stay, keep the weights (in registers, or for wider rows in shared memory) and
// copy the rows to come ahead of the one they work on, each thread its own
// pieces, so that no barrier guards them.
__device__ __forceinline__ float norm_block_sum(float v, float* red) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// Four values from 16 bytes of float32, or 8 of bf16.
__device__ __forceinline__ void norm_unpack(const uint4& v, float* f) {
  f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void norm_unpack(const uint2& v, float* f) {
  BF16::unpack2(v.x, f[0], f[1]);
  BF16::unpack2(v.y, f[2], f[3]);
}
template <class T>
struct NormPiece;
template <>
struct NormPiece<F32> {
  using Raw = uint4;
};
template <>
struct NormPiece<BF16> {
  using Raw = uint2;
};
template <class T>
__device__ __forceinline__ void norm_load4(const void* p, int64_t e, float* f) {
  norm_unpack(__ldcg(reinterpret_cast<const typename NormPiece<T>::Raw*>(static_cast<const char*>(p) + e * T::kBytes)), f);
}
template <class T>
__device__ __forceinline__ void norm_store4(void* p, int64_t e, const float* f) {
  if constexpr (T::kBytes == 2) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(static_cast<char*>(p) + e * 2) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(static_cast<char*>(p) + e * 4) = make_float4(f[0], f[1], f[2], f[3]);
  }
}
// Four float32 parameters (SHARED: staged in shared memory).
template <bool SHARED>
__device__ __forceinline__ float4 norm_param4(const float* p, int c) {
  if constexpr (SHARED) return *reinterpret_cast<const float4*>(p + c);
  else return __ldcg(reinterpret_cast<const float4*>(p + c));
}
// Where a norm's weight and bias come from: piece i, column c (absent: 1 and 0).
template <bool SHARED>
struct NormMem {
  const float *w, *b;
  __device__ __forceinline__ float4 weight(int, int c) const { return w ? norm_param4<SHARED>(w, c) : make_float4(1.f, 1.f, 1.f, 1.f); }
  __device__ __forceinline__ float4 bias(int, int c) const { return b ? norm_param4<SHARED>(b, c) : make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <int VPT>
struct NormRegs {
  float4 w[VPT], b[VPT];
  __device__ __forceinline__ void load(const float* wp, const float* bp, const int (&c)[VPT]) {
    const NormMem<false> m{wp, bp};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      w[i] = m.weight(i, c[i]);
      b[i] = m.bias(i, c[i]);
    }
  }
  __device__ __forceinline__ float4 weight(int i, int) const { return w[i]; }
  __device__ __forceinline__ float4 bias(int i, int) const { return b[i]; }
};

// A thread's pieces: their columns (those beyond the row stand on column 0 and
// count 0 in one[]; their values, which may be those of column 0's weight, bias
// and gate, never leave the thread).
template <int VPT>
struct NormRow {
  int c[VPT];
  float one[VPT], inv_d;
  __device__ __forceinline__ NormRow(int d) : inv_d(1.f / float(d)) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      c[i] = (threadIdx.x + i * blockDim.x) * 4;
      one[i] = c[i] < d ? 1.f : 0.f;
      if (c[i] >= d) c[i] = 0;
    }
  }
  __device__ __forceinline__ bool in(int i) const { return one[i] != 0.f; }
};

// v <- norm(v) * weight + bias over the row (on entry 0 beyond it); red: two rows of 32 sums.
template <int VPT, class P>
__device__ __forceinline__ void norm_row(float (&v)[VPT][4], int kind, float eps, const P& par, const NormRow<VPT>& k,
                                         float (*red)[32]) {
  if (kind == GSI_NORM_NONE) return;
  if (kind == GSI_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) s += (v[i][0] + v[i][1]) + (v[i][2] + v[i][3]);
    const float mean = norm_block_sum(s, red[0]) * k.inv_d;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = fmaf(-mean, k.one[i], v[i][e]);
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) q = fmaf(v[i][e], v[i][e], q);
  const float r = rsqrtf(fmaf(norm_block_sum(q, red[1]), k.inv_d, eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const float4 wv = par.weight(i, k.c[i]), bv = par.bias(i, k.c[i]);
    v[i][0] = fmaf(v[i][0] * r, wv.x, bv.x);
    v[i][1] = fmaf(v[i][1] * r, wv.y, bv.y);
    v[i][2] = fmaf(v[i][2] * r, wv.z, bv.z);
    v[i][3] = fmaf(v[i][3] * r, wv.w, bv.w);
  }
}

// One row from its values in y and h (0 beyond the row) to its stores.  gate:
// the token's row of the gate (in shared memory where SHARED_GATE);
// no_gate: a gate of 0.
template <class HT, class XT, int VPT, bool SHARED_GATE, class P>
__device__ __forceinline__ void norm_token(const NormArgs& a, const NormRow<VPT>& k, const P& post, const P& pre, int64_t row,
                                           float (&y)[VPT][4], float (&h)[VPT][4], const float* gate, bool no_gate,
                                           float (*red)[32]) {
  float4 gv[VPT];
  if (a.gate) {  // ahead of the reduction
#pragma unroll
    for (int i = 0; i < VPT; ++i) gv[i] = no_gate ? make_float4(0.f, 0.f, 0.f, 0.f) : norm_param4<SHARED_GATE>(gate, k.c[i]);
  }
  if (a.Y) {
    norm_row<VPT>(y, a.post, a.post_eps, post, k, red);
    if (a.gate) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) y[i][0] *= gv[i].x, y[i][1] *= gv[i].y, y[i][2] *= gv[i].z, y[i][3] *= gv[i].w;
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) h[i][e] = k.in(i) ? fmaf(a.alpha, h[i][e], y[i][e]) : 0.f;  // (an infinity times 0 is none)
  if (a.H_out) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (k.in(i)) norm_store4<HT>(a.H_out, row + k.c[i], h[i]);
  }
  if (!a.X) return;
  norm_row<VPT>(h, a.pre, a.pre_eps, pre, k, red + 2);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (k.in(i)) norm_store4<XT>(a.X, row + k.c[i], h[i]);
}

// A CTA a token.
template <class HT, class YT, class XT, int VPT>
__global__ void __launch_bounds__(1024, 1) norm_token_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[4][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x, row = t * a.d;
  const NormRow<VPT> k(a.d);
  float h[VPT][4] = {}, y[VPT][4] = {};
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (k.in(i)) {
      if (a.Y) norm_load4<YT>(a.Y, row + k.c[i], y[i]);
      norm_load4<HT>(a.H, row + k.c[i], h[i]);
    }
  const int g = a.gate && a.gate_index ? __ldcg(a.gate_index + t) : 0;
  norm_token<HT, XT, VPT, false>(a, k, NormMem<false>{a.post_w, a.post_b}, NormMem<false>{a.pre_w, a.pre_b}, row, y, h,
                                 a.gate + int64_t(g) * a.d, g < 0 || g >= a.gate_rows, red);
}

// CTAs that stay: tokens blockIdx.x, + gridDim.x, ...  Shared memory: a gate of
// one row, then kNormAhead + 1 rows' pieces, those of a thread written and read
// by it alone.  The weights are in registers (REGS, two pieces a thread, up to
// 5120 values), or, where wider rows leave no room for them, in shared memory
// before the rows (four pieces a thread): 2049 x 5120 LAYER takes 36 us (4.1
// TB/s) the first way and 42 us the second, whose fewer warps wait on each other
// longer.  What is left is the row's own chain, with one row in work a CTA: up to
// four reductions of ~400 cycles, and ~460 instructions a warp.  Staying CTAs and
// a CTA a token, us: 2049 x 5120 LAYER 37 and 56, RMS 33 and 44 (a gate a
// request each), 2049 x 5128 RMS (shared memory) 30 and 41, 2048 x 4096 LAYER 29
// and 52, 2048 x 6144 LAYER of bf16 rows 38 and 61.  Rows that neither form
// holds take a CTA a token: 2048 x 8192 LAYER 77, 2048 x 16384 125 (of 35 and 69
// us of bytes).
constexpr int kNormAhead = 3;
template <bool REGS>
struct NormRowsCfg {
  static constexpr int kVpt = REGS ? 2 : 4, kThreads = REGS ? 640 : 512;
};

template <int BYTES>
__device__ __forceinline__ void norm_copy(void* dst, const void* src) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(s), "l"(src) : "memory");
}

template <class HT, class YT, class XT, bool REGS>
__global__ void __launch_bounds__(NormRowsCfg<REGS>::kThreads, 1) norm_rows_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ uint4 norm_smem[];
  __shared__ float red[4][32];
  constexpr int VPT = NormRowsCfg<REGS>::kVpt;
  using Par = std::conditional_t<REGS, NormRegs<VPT>, NormMem<true>>;
  using RawY = typename NormPiece<YT>::Raw;
  using RawH = typename NormPiece<HT>::Raw;
  const int tid = threadIdx.x, nt = blockDim.x;
  pdl_launch_dependents();
  pdl_wait();
  float* par = reinterpret_cast<float*>(norm_smem);
  auto stage = [&](const float* p) -> const float* {
    if (!p) return nullptr;
    float* at = par;
    for (int c = tid * 4; c < a.d; c += nt * 4) norm_copy<16>(at + c, p + c);
    par += a.d;
    return at;
  };
  const NormRow<VPT> k(a.d);
  Par post, pre;
  if constexpr (REGS) {
    post.load(a.post_w, a.post_b, k.c);
    pre.load(a.pre_w, a.pre_b, k.c);
  } else {
    post = Par{stage(a.post_w), stage(a.post_b)};
    pre = Par{stage(a.pre_w), stage(a.pre_b)};
  }
  const bool by_index = a.gate && a.gate_index;
  const float* gate = by_index ? a.gate : stage(a.gate);
  RawY* ry = reinterpret_cast<RawY*>(par) + tid;                                     // [slot][piece][thread]
  RawH* rh = reinterpret_cast<RawH*>(reinterpret_cast<RawY*>(par) + (kNormAhead + 1) * VPT * nt) + tid;
  auto fetch = [&](int64_t t, int slot) {
    if (t < a.T) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (k.in(v)) {
          if (a.Y) norm_copy<sizeof(RawY)>(ry + (slot * VPT + v) * nt, static_cast<const char*>(a.Y) + (t * a.d + k.c[v]) * YT::kBytes);
          norm_copy<sizeof(RawH)>(rh + (slot * VPT + v) * nt, static_cast<const char*>(a.H) + (t * a.d + k.c[v]) * HT::kBytes);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t t = blockIdx.x;
  const int64_t step = gridDim.x;
#pragma unroll
  for (int i = 0; i < kNormAhead; ++i) fetch(t + i * step, i);
  int g = by_index ? __ldcg(a.gate_index + t) : 0;
  for (int it = 0; t < a.T; ++it, t += step) {
    fetch(t + kNormAhead * step, (it + kNormAhead) & kNormAhead);
    const int g_next = by_index && t + step < a.T ? __ldcg(a.gate_index + t + step) : 0;
    asm volatile("cp.async.wait_group %0;" ::"n"(kNormAhead) : "memory");  // (the parameters are in the first group)
    __syncthreads();  // the parameters of every thread are there; the sums of the row before have been read
    float y[VPT][4] = {}, h[VPT][4] = {};
    const int slot = it & kNormAhead;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (k.in(v)) {
        if (a.Y) norm_unpack(ry[(slot * VPT + v) * nt], y[v]);
        norm_unpack(rh[(slot * VPT + v) * nt], h[v]);
      }
    if (by_index)
      norm_token<HT, XT, VPT, false>(a, k, post, pre, t * a.d, y, h, gate + int64_t(g) * a.d, g < 0 || g >= a.gate_rows, red);
    else
      norm_token<HT, XT, VPT, true>(a, k, post, pre, t * a.d, y, h, gate, false, red);
    g = g_next;
  }
}
static_assert((kNormAhead & (kNormAhead + 1)) == 0, "a slot is the row's number modulo a power of two");

// false: this form does not hold the row.
template <class HT, class YT, class XT, bool REGS>
static bool launch_norm_rows(const NormArgs& a, cudaLaunchConfig_t cfg, cudaError_t* e) {
  using C = NormRowsCfg<REGS>;
  const int threads = ((a.d / 4 + C::kVpt - 1) / C::kVpt + 31) / 32 * 32;
  const int params = (!REGS && a.post_w) + (!REGS && a.post_b) + (!REGS && a.pre_w) + (!REGS && a.pre_b) +
                     (a.gate && !a.gate_index);
  const size_t smem = size_t(params) * a.d * 4 + size_t(kNormAhead + 1) * C::kVpt * threads * 4 * (HT::kBytes + YT::kBytes);
  constexpr size_t kMost = 232448 - 1024;
  if (threads > C::kThreads || smem > kMost) return false;
  static OnEveryDevice ready;
  *e = ready([] {
    return cudaFuncSetAttribute(norm_rows_kernel<HT, YT, XT, REGS>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost));
  });
  if (*e != cudaSuccess) return true;
  // CTAs of an SM: what its registers and shared memory hold
  const int per_sm = max(1, min(C::kThreads / threads, int(kMost / (smem + 2048))));
  cfg.gridDim = dim3(min(a.T, sm_count() * per_sm));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  *e = cudaLaunchKernelEx(&cfg, norm_rows_kernel<HT, YT, XT, REGS>, a);
  return true;
}

template <class HT, class YT, class XT>
static cudaError_t launch_norm_types(const NormArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // CTAs that stay pay from the second token of an SM on (200 x 5120 LAYER: 5.8 us, a CTA a token 6.5; 303: 5.9 and 6.7)
  cudaError_t e;
  if (a.T > sm_count() && (launch_norm_rows<HT, YT, XT, true>(a, cfg, &e) || launch_norm_rows<HT, YT, XT, false>(a, cfg, &e)))
    return e;
  const int pieces = a.d / 4;
  const auto threads_for = [&](int vpt) { return ((pieces + vpt - 1) / vpt + 31) / 32 * 32; };
  cfg.gridDim = dim3(a.T);
  const int vpt = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
  cfg.blockDim = dim3(threads_for(vpt));
  switch (vpt) {
    case 1: return cudaLaunchKernelEx(&cfg, norm_token_kernel<HT, YT, XT, 1>, a);
    case 2: return cudaLaunchKernelEx(&cfg, norm_token_kernel<HT, YT, XT, 2>, a);
    default: return cudaLaunchKernelEx(&cfg, norm_token_kernel<HT, YT, XT, 4>, a);
  }
}

cudaError_t launch_norm_residual(const NormArgs& a, gsi_dtype hdt, gsi_dtype ydt, gsi_dtype xdt, cudaStream_t s) {
  const int which = (hdt == GSI_BF16) * 4 + (ydt == GSI_BF16) * 2 + (xdt == GSI_BF16);
  switch (which) {
    case 0: return launch_norm_types<F32, F32, F32>(a, s);
    case 1: return launch_norm_types<F32, F32, BF16>(a, s);
    case 2: return launch_norm_types<F32, BF16, F32>(a, s);
    case 3: return launch_norm_types<F32, BF16, BF16>(a, s);
    case 4: return launch_norm_types<BF16, F32, F32>(a, s);
    case 5: return launch_norm_types<BF16, F32, BF16>(a, s);
    case 6: return launch_norm_types<BF16, BF16, F32>(a, s);
    default: return launch_norm_types<BF16, BF16, BF16>(a, s);
  }
}

}  // namespace gsi
