// The end of one block and the beginning of the next in one pass:
//   h' = alpha h + gate * post(y),   x = pre(h').

#include "gsi_common.cuh"
#include "gsi_kernels.h"

namespace gsi {

// One CTA a token.  Every value of the row stays in registers from its load
// to its stores: y and h are read once, h' and x written once, and the norms'
// sums are block reductions between (LAYER: the mean first, then the centred
// squares, so no difference of large sums).  The bytes bound it at prompt
// sizes; one token is a chain of loads and up to four reductions.
template <int N>
__device__ __forceinline__ float norm_block_sum(float v, float* red) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
  s = warp_sum(s);
  return s;
}

template <class T>
__device__ __forceinline__ void norm_load8(const void* p, int64_t e, float* f) {
  if constexpr (T::kBytes == 2) {
    T::unpack(ld_cg_v4(static_cast<const char*>(p) + e * 2), f);
  } else {
    T::unpack(ld_cg_v4(static_cast<const char*>(p) + e * 4), f);
    T::unpack(ld_cg_v4(static_cast<const char*>(p) + e * 4 + 16), f + 4);
  }
}

template <class T>
__device__ __forceinline__ void norm_store8(void* p, int64_t e, const float* f) {
  if constexpr (T::kBytes == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(static_cast<char*>(p) + e * 2) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<char*>(p) + e * 4);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// v <- norm(v) * weight + bias over the row (VPT vectors of 8 a thread; red:
// two rows of 32 partial sums).
template <int VPT>
__device__ __forceinline__ void norm_row(float (&v)[VPT][8], int kind, float eps, const float* w, const float* b, int d,
                                         float (*red)[32]) {
  if (kind == GSI_NORM_NONE) return;
  if (kind == GSI_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[i][e];
    const float mean = norm_block_sum<VPT>(s, red[0]) / float(d);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if ((threadIdx.x + i * blockDim.x) * 8 < d)
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(v[i][e], v[i][e], q);
  const float r = rsqrtf(norm_block_sum<VPT>(q, red[1]) / float(d) + eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c >= d) continue;
    float wv[8], bv[8];
    if (w) norm_load8<F32>(w, c, wv);
    if (b) norm_load8<F32>(b, c, bv);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[i][e] *= r;
      if (w) v[i][e] *= wv[e];
      if (b) v[i][e] += bv[e];
    }
  }
}

template <class HT, class YT, class XT, int VPT>
__global__ void __launch_bounds__(1024) norm_residual_kernel(NormArgs a) {
  __shared__ float red[4][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int64_t row = t * a.d;
  float h[VPT][8], y[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = y[i][e] = 0.f;
    if (c < a.d) {
      if (a.Y) norm_load8<YT>(a.Y, row + c, y[i]);
      norm_load8<HT>(a.H, row + c, h[i]);
    }
  }
  int64_t g = 0;
  if (a.gate && a.gate_index) g = __ldcg(a.gate_index + t);
  if (a.Y) norm_row<VPT>(y, a.post, a.post_eps, a.post_w, a.post_b, a.d, red);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c >= a.d) continue;
    float gv[8];
    if (a.gate) {
#pragma unroll
      for (int e = 0; e < 8; ++e) gv[e] = 0.f;
      if (g >= 0 && g < a.gate_rows) norm_load8<F32>(a.gate, g * a.d + c, gv);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float u = a.alpha * h[i][e];
      if (a.Y) u = a.gate ? fmaf(gv[e], y[i][e], u) : u + y[i][e];
      h[i][e] = u;
    }
    if (a.H_out) norm_store8<HT>(a.H_out, row + c, h[i]);
  }
  if (!a.X) return;
  norm_row<VPT>(h, a.pre, a.pre_eps, a.pre_w, a.pre_b, a.d, red + 2);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c < a.d) norm_store8<XT>(a.X, row + c, h[i]);
  }
}

template <class HT, class YT, class XT>
static cudaError_t launch_norm_types(const NormArgs& a, cudaStream_t s) {
  const int n_vec = a.d / 8;
  const int vpt = n_vec > 1024 ? 2 : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.T);
  cfg.blockDim = dim3(((n_vec + vpt - 1) / vpt + 31) / 32 * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return vpt == 2 ? cudaLaunchKernelEx(&cfg, norm_residual_kernel<HT, YT, XT, 2>, a)
                  : cudaLaunchKernelEx(&cfg, norm_residual_kernel<HT, YT, XT, 1>, a);
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
