// Attention over a float32 cache, on the CUDA cores: the tensor cores have no
// float32 product, and the next best (tf32) keeps 11 bits.

#include "gsi_attn.cuh"

namespace gsi {

// A unit is BM query rows over tiles of 64 keys: S = Q K^T and O += P V as
// register tiles of 256 threads, the keys and values of a tile copied into
// shared memory while the other product runs (V during S, the next K during
// O).  A row's 64 scores lie in TK lanes of one warp, so its maximum and sum
// are shuffles and P only passes through the warp's own rows of shared memory.
//   BM = 64: 4 x 4 scores a thread; 64 fused products for 8 vector loads of
//            shared memory, so the FMA pipes bound it (74 TFLOP/s of the SMs);
//   BM = 16: 2 x 2, for few rows: 16 rows' products keep up with the bytes.
// Values a masked tile hides are set to zero in shared memory as they arrive
// where no row sees their key, and where they are not finite (added at the end
// for the rows that do see them).
// 2048 tokens of 16 x 64: 317 us, 27 TFLOP/s of what the mask leaves; one token
// over 100,000 keys of 8 x 128: 372 us, 2.2 TB/s (the shared-memory loads of 2 x 2
// tiles).
constexpr int kF32Keys = 64, kF32Threads = 256;

template <int BM>
struct F32Cfg {
  static constexpr int kTK = BM == 64 ? 16 : 32;      // lanes of a row group
  static constexpr int kRM = BM == 64 ? 4 : 2;        // rows of a group
  static constexpr int kKN = kF32Keys / kTK;          // keys a thread scores
  static constexpr int kPStride = kF32Keys + 4;
  static_assert(kF32Threads / kTK * kRM == BM, "rows");
  static size_t smem(int dim) { return (size_t(BM + 2 * kF32Keys) * (dim + 4) + size_t(BM) * kPStride) * 4; }
};

__device__ __forceinline__ void f32_copy16(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sa(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void f32_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void f32_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <int BM, int NC>  // NC: 4-column pieces of the output a thread holds of each row
__global__ void __launch_bounds__(kF32Threads, BM == 16 || NC <= 2 ? 2 : 1) attn_f32_kernel(const __grid_constant__ AttnArgs a) {
  using C = F32Cfg<BM>;
  constexpr int TK = C::kTK, RM = C::kRM, KN = C::kKN, PS = C::kPStride;
  extern __shared__ __align__(16) float f32_smem[];
  __shared__ int s_last, s_found;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tk = tid % TK, tr = tid / TK;
  const int DP = a.dim + 4, d4 = a.dim / 4;
  float* sq = f32_smem;
  float* sk = sq + BM * DP;
  float* sv = sk + kF32Keys * DP;
  float* sp = sv + kF32Keys * DP;
  // the output's columns: CG lanes a row, the lanes left over take a part of the keys each
  // (four keys at a time, so at least TK / 16 lanes a row)
  int cg = TK / 16;
  while (cg < d4 && cg < TK) cg *= 2;
  const int kq = tk / cg, keys_each = kF32Keys * cg / TK, c0 = tk % cg;

  pdl_launch_dependents();
  if (tid == 0) s_found = 0;
  pdl_wait();
  AttnWalk walk;
  const int ut = walk.ut = BM / a.group;
  walk.kt = kF32Keys;
  walk.s = attn_share<kF32Threads>(a, ut, kF32Keys, 0, walk.p);
  AttnSeg g;
  while (walk.next(a, g)) {
    const int tok0 = g.u * ut, n_tok = min(ut, g.q.q_len - tok0), n_rows = n_tok * a.group;
    const int lim_all = attn_lim(a, g.q, tok0 + n_tok - 1), lim_min = attn_lim(a, g.q, tok0);
    const int lo_all = attn_lo(a, lim_min), lo_max = attn_lo(a, lim_all);
    // a tile's rows of K or V: warp w copies 8 of them
    auto copy = [&](float* dst, const void* src, int i) {
      const int key = (g.t0 + i) * kF32Keys + warp * 8 + (lane & 7);
      long long at = -1;
      if (key >= lo_all && key < lim_all) {
        const int pg = __ldcg(a.table + int64_t(g.r) * a.width + (key >> a.page_shift));
        if (pg >= 0 && pg < a.n_pages)
          at = pg * a.page_stride + g.h * a.head_stride + int64_t(key & ((1 << a.page_shift) - 1)) * a.token_stride;
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const long long from = __shfl_sync(0xffffffffu, at, r);
        for (int c = lane; c < d4; c += 32)
          f32_copy16(dst + (warp * 8 + r) * DP + 4 * c, static_cast<const float*>(src) + (from < 0 ? 0 : from) + 4 * c, from >= 0);
      }
      f32_commit();
    };
    if (g.b > g.a) copy(sk, a.K, g.a);
    // weights are 2^(c (s - m)): the difference first, which is exact where it matters, and c > 0 (a negative scale
    // turns q over, a scale of 0 still masks)
    const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f), sign = a.scale < 0.f ? -1.f : 1.f;
    for (int e = tid; e < BM * d4; e += kF32Threads) {
      const int row = e / d4, x = e - row * d4, tok = row / a.group;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < n_rows)
        v = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(a.Q) + int64_t(g.q.q0 + tok0 + tok) * a.q_stride +
                                                   int64_t(g.h * a.group + row - tok * a.group) * a.dim) + x);
      *reinterpret_cast<float4*>(sq + row * DP + 4 * x) = make_float4(v.x * sign, v.y * sign, v.z * sign, v.w * sign);
    }
    int lim[RM], lo[RM];
    float m[RM], l[RM], o[RM][NC][4];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int row = tr * RM + i;
      lim[i] = row < n_rows ? attn_lim(a, g.q, tok0 + row / a.group) : 0;
      lo[i] = attn_lo(a, lim[i]);
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int n = 0; n < NC; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
    for (int j = g.a; j < g.b; ++j) {
      f32_wait_all();
      __syncthreads();  // K is there (and Q); the product before is done with V
      copy(sv, a.V, j);
      float s[RM][KN];
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int n = 0; n < KN; ++n) s[i][n] = 0.f;
#pragma unroll 4
      for (int x = 0; x < d4; ++x) {
        float4 q[RM], k[KN];
#pragma unroll
        for (int i = 0; i < RM; ++i) q[i] = *reinterpret_cast<const float4*>(sq + (tr * RM + i) * DP + 4 * x);
#pragma unroll
        for (int n = 0; n < KN; ++n) k[n] = *reinterpret_cast<const float4*>(sk + (tk + n * TK) * DP + 4 * x);
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
          for (int n = 0; n < KN; ++n)
            s[i][n] = fmaf(q[i].w, k[n].w, fmaf(q[i].z, k[n].z, fmaf(q[i].y, k[n].y, fmaf(q[i].x, k[n].x, s[i][n]))));
      }
      const int tile = (g.t0 + j) * kF32Keys;
      const bool partial = tile < lo_max || tile + kF32Keys > lim_min;
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        if (partial) {
#pragma unroll
          for (int n = 0; n < KN; ++n) {
            const int key = tile + tk + n * TK;
            if (key < lo[i] || key >= lim[i]) s[i][n] = -INFINITY;
          }
        }
        float mx = m[i];
#pragma unroll
        for (int n = 0; n < KN; ++n) mx = fmaxf(mx, s[i][n]);
#pragma unroll
        for (int b = TK / 2; b > 0; b >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, b));
        const float f = m[i] == -INFINITY ? 0.f : ex2((m[i] - mx) * c), to = mx == -INFINITY ? 0.f : mx;
        m[i] = mx;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < KN; ++n) {
          const float p = ex2((s[i][n] - to) * c);
          sum += p;
          sp[(tr * RM + i) * PS + tk + n * TK] = p;
        }
        l[i] = l[i] * f + sum;  // this lane's keys
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][n][e] *= f;
      }
      f32_wait_all();
      __syncthreads();  // V is there, and P; every thread is done with K
      if (j + 1 < g.b) copy(sk, a.K, j + 1);
      if (partial) {
        bool found = false;
        for (int e = tid; e < kF32Keys * d4; e += kF32Threads) {
          float4* v = reinterpret_cast<float4*>(sv + e / d4 * DP) + e % d4;
          float4 w = *v;
          bool bad = false;
          if (!(fabsf(w.x) < INFINITY)) w.x = 0.f, bad = true;
          if (!(fabsf(w.y) < INFINITY)) w.y = 0.f, bad = true;
          if (!(fabsf(w.z) < INFINITY)) w.z = 0.f, bad = true;
          if (!(fabsf(w.w) < INFINITY)) w.w = 0.f, bad = true;
          if (bad) *v = w;
          found |= bad;
        }
        if (found) s_found = 1;
        __syncthreads();
      }
      for (int k = kq * keys_each; k < (kq + 1) * keys_each; k += 4) {
        float4 p[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (tr * RM + i) * PS + k);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const int col = c0 + n * cg;
          if (col >= d4) break;
          const float* v0 = sv + k * DP + 4 * col;
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float4 v = *reinterpret_cast<const float4*>(v0 + z * DP);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
              const float w = z == 0 ? p[i].x : z == 1 ? p[i].y : z == 2 ? p[i].z : p[i].w;
              o[i][n][0] = fmaf(w, v.x, o[i][n][0]);
              o[i][n][1] = fmaf(w, v.y, o[i][n][1]);
              o[i][n][2] = fmaf(w, v.z, o[i][n][2]);
              o[i][n][3] = fmaf(w, v.w, o[i][n][3]);
            }
          }
        }
      }
    }
    // ---- the segment's end: a row's sum over its lanes, its output over the lanes with the same columns
#pragma unroll
    for (int i = 0; i < RM; ++i) {
#pragma unroll
      for (int b = TK / 2; b > 0; b >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], b);
      for (int b = cg; b < TK; b *= 2)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][n][e] += __shfl_xor_sync(0xffffffffu, o[i][n][e], b);
    }
    __syncthreads();  // every tile's `found`
    const bool any = s_found != 0;
    const bool whole = g.a == 0 && g.b == g.n;
    int b0, b1;
    walk.parts(g, b0, b1);
    float* part = attn_part(a, 2 * int(blockIdx.x) + (int(blockIdx.x) == b0), 1, 0, BM);
    if (kq == 0) {
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const int row = tr * RM + i;
        if (row >= n_rows) continue;
        const float inv = !whole ? 1.f : l[i] != 0.f ? 1.f / l[i] : lim[i] > 0 ? NAN : 0.f;  // as attn_inverse
        if (!whole && c0 == 0) {
          part[row] = m[i] == -INFINITY ? m[i] : m[i] * c;
          part[BM + row] = l[i];
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const int col = c0 + n * cg;
          if (col >= d4) continue;
          if (any)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[i][n][e] = attn_nonfinite<F32>(a, g, kF32Keys, lo[i], lim[i], lo_max, lim_min, 4 * col + e, o[i][n][e]);
          const float4 v = make_float4(o[i][n][0] * inv, o[i][n][1] * inv, o[i][n][2] * inv, o[i][n][3] * inv);
          if (whole)
            *reinterpret_cast<float4*>(static_cast<float*>(a.O) + attn_out_row(a, g, tok0, row) * a.dim + 4 * col) = v;
          else
            *attn_piece<true>(part, BM, a.dim, row, 4 * col) = v;
        }
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned n = unsigned(b1 - b0 + 1);
        const bool last = atomicAdd(attn_counter(a, b0, 0), 1u) == n - 1;
        if (last) *attn_counter(a, b0, 0) = 0;
        s_last = last;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        attn_join<F32, true, 4>(a, g, b0, b1, 1, 0, BM, n_rows, tok0, tid, kF32Threads);
      }
    }
    __syncthreads();  // before the next segment writes Q and the flags
    if (tid == 0) s_found = 0;
  }
}

template <int BM, int NC>
static cudaError_t launch_f32(const AttnArgs& a, cudaStream_t s) {
  static OnEveryDevice ready;
  const cudaError_t e = ready([] { return attn_prepare_kernel(attn_f32_kernel<BM, NC>, F32Cfg<BM>::smem(256), kF32Threads, 0); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const size_t smem = F32Cfg<BM>::smem(a.dim);
  const int per_sm = (BM == 16 || NC <= 2) && 2 * (smem + 2048) <= 233472 ? 2 : 1;  // CTAs that an SM holds
  cfg.gridDim = dim3(per_sm * min(sm_count(), kAttnCtas));
  cfg.blockDim = dim3(kF32Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_f32_kernel<BM, NC>, a);
}

cudaError_t launch_attn_f32(const AttnArgs& a, bool few, cudaStream_t s) {
  if (few) return a.dim <= 128 ? launch_f32<16, 1>(a, s) : launch_f32<16, 2>(a, s);
  switch ((a.dim + 63) / 64) {
    case 1: return launch_f32<64, 1>(a, s);
    case 2: return launch_f32<64, 2>(a, s);
    case 3: return launch_f32<64, 3>(a, s);
    default: return launch_f32<64, 4>(a, s);
  }
}

}  // namespace gsi
