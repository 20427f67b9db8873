// Accumulated attention weights of cached keys: dispatch, and the kernel on the
// CUDA cores.

#include <algorithm>

#include "gsi_weights.cuh"

namespace gsi {

// A unit is 64 keys, a step up to 64 query rows at a time (few rows: 16): scores
// as register tiles of 4 x 4 (4 x 1) over 256 threads, keys and rows in shared
// memory as float32; a thread adds its rows' weights to its four keys' sums, and
// the sixteen row groups are added when the part of the unit ends, in one order.
// Up to four CTAs an SM, so that one's loads pass under another's products
// (few rows, where that is what bounds them: one token of 16 requests of 2048
// keys, 16 x 128, 395 us with one CTA, all of its rows formed whether there or not,
// 109 with three, 88 with four and a spill of 68 bytes; 1.8 TB/s).  The score, its
// scaling and the row's logarithm meet in one fused product, exact up to its
// result, so a weight's error is that of its score.
constexpr int kKwKeys = 64, kKwThreads = 256;

template <class T, int RM>
__global__ void __launch_bounds__(kKwThreads, RM == 1 ? 4 : 2) key_weights_kernel(const __grid_constant__ KeyWeightArgs a, int tpt) {
  constexpr int kKwRows = 16 * RM;
  extern __shared__ __align__(16) float kw_smem[];
  __shared__ float s_sum[kKwThreads / 32][kKwKeys];
  __shared__ float s_lse[kKwRows];
  __shared__ float s_part[RM == 1 ? 16 : 1][kKwKeys];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tk = tid % 16, tr = tid / 16;
  const int DP = a.dim + 4, d4 = a.dim / 4, vec = a.dim / T::kPerVec;
  float* sk = kw_smem;
  float* sq = sk + kKwKeys * DP;
  pdl_launch_dependents();
  pdl_wait();
  KwWalk<kKwKeys> walk;
  kw_share<kKwKeys, kKwThreads>(a, tpt, walk);
  KwSeg g;
  while (walk.next(a, g)) {
    const int key0 = g.t * kKwKeys;
    float acc[4] = {};
    if (g.q.q_len > 0) {
      for (int e = tid; e < kKwKeys * vec; e += kKwThreads) {
        const int row = e / vec, c = (e - row * vec) * T::kPerVec, key = key0 + row;
        float v[T::kPerVec] = {};
        if (key < g.q.len) {
          const int pg = __ldcg(a.table + int64_t(g.r) * a.width + (key >> a.page_shift));
          if (pg >= 0 && pg < a.n_pages)
            T::unpack(ld_cg_v4(static_cast<const char*>(a.K) +
                               (pg * a.page_stride + g.h * a.head_stride +
                                int64_t(key & ((1 << a.page_shift) - 1)) * a.token_stride + c) * T::kBytes), v);
        }
#pragma unroll
        for (int x = 0; x < T::kPerVec; ++x) sk[row * DP + c + x] = v[x];
      }
      const int per_step = (tpt * a.group + kKwRows - 1) / kKwRows;
      for (int u = (g.u0 + g.a) * per_step; u < (g.u0 + g.b) * per_step; ++u) {
        const int tok0 = u / per_step * tpt, row0 = u % per_step * kKwRows;
        const int n_rows = min(kKwRows, min(tpt, g.q.q_len - tok0) * a.group - row0);
        if (n_rows <= 0) continue;
        __syncthreads();  // the rows before have been used
        for (int e = tid; e < kKwRows * vec; e += kKwThreads) {
          const int row = e / vec, c = (e - row * vec) * T::kPerVec;
          float v[T::kPerVec] = {};
          if (row < n_rows) {
            const int tok = (row0 + row) / a.group, head = g.h * a.group + (row0 + row) % a.group;
            T::unpack(ld_cg_v4(static_cast<const char*>(a.Q) +
                               (int64_t(g.q.q0 + tok0 + tok) * a.q_stride + int64_t(head) * a.dim + c) * T::kBytes), v);
          }
#pragma unroll
          for (int x = 0; x < T::kPerVec; ++x) sq[row * DP + c + x] = v[x];
        }
        if (tid < n_rows) {
          const int tok = (row0 + tid) / a.group, head = g.h * a.group + (row0 + tid) % a.group;
          s_lse[tid] = __ldcg(a.LSE + int64_t(g.q.q0 + tok0 + tok) * a.hkv * a.group + head);
        }
        __syncthreads();
        // few rows: the row groups that are left over take a part of the columns each (a row's products in 16 / R parts, R the
        // power of two from its rows on)
        const int rows2 = RM > 1 || n_rows > 8 ? 16 : n_rows > 4 ? 8 : n_rows > 2 ? 4 : n_rows;
        const int parts = RM > 1 ? 1 : 16 / rows2, mine = RM > 1 ? tr : tr % rows2, part = RM > 1 ? 0 : tr / rows2;
        float s[RM][4] = {};
#pragma unroll 4
        for (int x = d4 * part / parts; x < d4 * (part + 1) / parts; ++x) {
          float4 q[RM], k[4];
#pragma unroll
          for (int i = 0; i < RM; ++i) q[i] = *reinterpret_cast<const float4*>(sq + (mine * RM + i) * DP + 4 * x);
#pragma unroll
          for (int n = 0; n < 4; ++n) k[n] = *reinterpret_cast<const float4*>(sk + (tk + 16 * n) * DP + 4 * x);
#pragma unroll
          for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n)
              s[i][n] = fmaf(q[i].w, k[n].w, fmaf(q[i].z, k[n].z, fmaf(q[i].y, k[n].y, fmaf(q[i].x, k[n].x, s[i][n]))));
        }
        if (parts > 1) {
#pragma unroll
          for (int n = 0; n < 4; ++n) s_part[tr][tk + 16 * n] = s[0][n];
          __syncthreads();
          if (part == 0)
            for (int z = 1; z < parts; ++z)
#pragma unroll
              for (int n = 0; n < 4; ++n) s[0][n] += s_part[mine + z * rows2][tk + 16 * n];
        }
#pragma unroll
        for (int i = 0; i < RM; ++i) {
          const int row = mine * RM + i;
          if (row >= n_rows || part > 0) break;
          const int lim = a.causal ? g.q.len - g.q.q_len + tok0 + (row0 + row) / a.group + 1 : g.q.len;
          const float lse = s_lse[row];
#pragma unroll
          for (int n = 0; n < 4; ++n)
            if (key0 + tk + 16 * n < lim) acc[n] += exp2f(fmaf(s[i][n], a.scale, -lse) * 1.4426950408889634f);
        }
      }
    }
    // ---- the part's end: the sixteen row groups
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      acc[n] += __shfl_xor_sync(0xffffffffu, acc[n], 16);
      if (lane < 16) s_sum[warp][tk + 16 * n] = acc[n];
    }
    __syncthreads();
    float sum = 0.f;
    if (tid < kKwKeys)
#pragma unroll
      for (int w = 0; w < kKwThreads / 32; ++w) sum += s_sum[w][tid];
    if (g.a == 0 && g.b == g.n) {
      if (tid < kKwKeys) kw_give(a, g, key0 + tid, kw_mark(a, g, key0 + tid), sum);
    } else {
      int b0, b1;
      walk.parts(g, b0, b1);
      if (tid < kKwKeys) kw_part(a, 2 * int(blockIdx.x) + (int(blockIdx.x) == b0))[tid] = sum;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const bool last = atomicAdd(kw_counter(a, b0), 1u) == unsigned(b1 - b0);
        if (last) *kw_counter(a, b0) = 0;
        s_last = last;
      }
      __syncthreads();
      if (s_last && tid < kKwKeys) {
        __threadfence();
        sum = 0.f;
        for (int b = b0; b <= b1; ++b) sum += __ldcg(kw_part(a, 2 * b + (b == b0)) + tid);
        kw_give(a, g, key0 + tid, kw_mark(a, g, key0 + tid), sum);
      }
    }
    __syncthreads();  // before the next part writes the shared rows
  }
}

size_t key_weights_work_bytes() { return (kw_work_bytes() + 255) / 256 * 256; }

template <class T, int RM>
static cudaError_t launch_kw(const KeyWeightArgs& a, cudaStream_t s) {
  constexpr int kRows = 16 * RM;
  static OnEveryDevice ready;
  const cudaError_t e = ready([] {
    return cudaFuncSetAttribute(key_weights_kernel<T, RM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (kKwKeys + kRows) * 260 * 4);
  });
  if (e != cudaSuccess) return e;
  int tpt = 1;
  while (2 * tpt * a.group <= kRows) tpt *= 2;
  const size_t smem = size_t(kKwKeys + kRows) * (a.dim + 4) * 4;
  // One CTA an SM where that gives each two steps at most: units are cut less (64 tokens over 600 keys, 3 requests of 4 x 64:
  // 10.2 us, with two an SM 12.3; but 256 over 2048, 4 requests, 57 and 44).  `steps` is what they would be if rows filled
  // them and every request had the table's length.
  const int64_t steps = std::max<int64_t>(int64_t(a.N) * a.group / kRows + 1, a.n_req) * a.hkv * ((a.width << a.page_shift) / kKwKeys + 1);
  const int per_sm = steps <= 2 * sm_count() ? 1 : min(RM == 1 ? 4 : 2, int(233472 / (smem + 6144)));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(min(per_sm * sm_count(), kKwCtas));
  cfg.blockDim = dim3(kKwThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<T, RM>, a, tpt);
}

cudaError_t launch_key_weights(const KeyWeightArgs& a, gsi_dtype dt, int64_t max_q, cudaStream_t s) {
  if (a.N == 0) return dt == GSI_F32 ? launch_kw<F32, 1>(a, s) : launch_kw<BF16, 1>(a, s);  // keys to begin at zero, without a row
  // (the hint is the caller's: a step of 16 rows has to hold a token's heads)
  const bool few = std::clamp<int64_t>(max_q, 1, a.N) * a.group <= 16;
  if (dt == GSI_F32) return few ? launch_kw<F32, 1>(a, s) : launch_kw<F32, 4>(a, s);
  return launch_key_weights_tiles(a, few, s);
}

}  // namespace gsi
