// Attention of few query rows (decode): all rows of a unit in one 16-row
// tensor-core tile, the keys and values streamed once.

#include "gsi_attn.cuh"

namespace gsi {

// With G = group query heads a key/value head and ut = floor(16 / G) tokens a
// unit, S = Q K^T and O = P V have at most 16 rows: 16 FLOP a byte of cache,
// far below what the warp-level tensor products sustain, so the bytes bound
// the kernel and its work is to keep them coming.  One CTA an SM; a copy warp
// keeps a ring of 192 KB filled (64 keys and their values a stage, one TMA box
// a page and 64 columns, each lane issuing its own boxes); four warps take 16
// keys of each stage, each with a softmax of its own (running maximum m, sum
// l), joined when the CTA's part of a unit ends.  The scores' fragment of
// m16n8k16 is the next product's left operand as it stands, so P never leaves
// the registers.
constexpr int kRowsKt = 64;       // keys a stage
constexpr int kRowsWarps = 4;     // compute warps
constexpr int kRowsThreads = 32 * (kRowsWarps + 1);

template <int NS>  // 64-column slabs of a row
struct RowsCfg {
  static constexpr int kSlab = kRowsKt * 128;            // bytes
  static constexpr int kStage = 2 * NS * kSlab;          // K slabs, then V slabs
  static constexpr int kStages = 12 / NS;                // 192 KB
  static constexpr int kDim = NS * 64;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 16 * kDim * 4 + kRowsWarps * 32 * 4 + 2 * kStages * 8 + 16;
};

__device__ __forceinline__ void rows_ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void rows_ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void rows_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The compute warps only.
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kRowsWarps * 32) : "memory"); }

// A pair of bf16 values of keys j and j + 1: zero where the key lies outside
// [lo, lim) or the value is not finite (then *found is set).
__device__ __forceinline__ uint32_t rows_clean(uint32_t v, int j, int lo, int lim, bool& found) {
  uint32_t keep = 0;
  if (j >= lo && j < lim) {
    if ((v & 0x7f80u) != 0x7f80u) keep |= 0xffffu; else found = true;
  }
  if (j + 1 >= lo && j + 1 < lim) {
    if ((v & 0x7f800000u) != 0x7f800000u) keep |= 0xffff0000u; else found = true;
  }
  return v & keep;
}

template <int NS>
__global__ void __launch_bounds__(kRowsThreads, 1)
    attn_rows16_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ AttnArgs a) {
  using C = RowsCfg<NS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_o = reinterpret_cast<float*>(ring + size_t(C::kStages) * C::kStage);  // [16][kDim]
  float* s_ml = s_o + 16 * C::kDim;                                            // [warps][m: 16, l: 16]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ml + kRowsWarps * 32);
  uint64_t* empty = full + C::kStages;
  int* s_flag = reinterpret_cast<int*>(empty + C::kStages);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], kRowsWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mk) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mv) : "memory");
    s_flag[1] = 0;
  }
  pdl_wait();
  const int ut = 16 / a.group;
  const AttnShare share = attn_share<kRowsThreads>(a, ut, kRowsKt, 0);  // also publishes the barriers to the block
  AttnWalk walk;
  walk.begin(a, share, ut, kRowsKt);
  uint32_t* err = attn_err(a);
  AttnSeg g;
  int it = 0;  // stages so far

  if (warp == kRowsWarps) {
    // ---- copy warp: lane l issues box l of a stage (2 NS slabs of at most 4 boxes)
    const int page = 1 << a.page_shift;
    const int box = min(page, kRowsKt), boxes = kRowsKt / box;  // tokens of a box; boxes of a slab
    const uint32_t box_bytes = uint32_t(box) * 128;
    bool ok = true;
    while (ok && walk.next(a, g)) {
      const int lim_all = attn_lim(a, g.q, min((g.u + 1) * ut, g.q.q_len) - 1);
      const int lo_all = attn_lo(a, attn_lim(a, g.q, g.u * ut));
      const int32_t* row = a.table + int64_t(g.r) * a.width;
      for (int i = g.a; i < g.b; ++i, ++it) {
        const int s = it % C::kStages;
        const int key0 = (g.t0 + i) * kRowsKt;
        // only boxes with a key that some row sees
        const int first = max(lo_all - key0, 0) / box, last = min((lim_all - key0 + box - 1) / box, boxes);
        const int b = lane % boxes, slab = lane / boxes;  // this lane's box: slabs of K, then of V
        const bool mine = slab < 2 * NS && b >= first && b < last;
        const int pid = mine ? __ldcg(row + ((key0 + b * box) >> a.page_shift)) : 0;
        if (it >= C::kStages)
          ok = __all_sync(0xffffffffu, bar_wait(&empty[s], uint32_t(it / C::kStages - 1) & 1u, err));
        if (!ok) break;
        if (lane == 0) bar_expect_tx(&full[s], uint32_t(last - first) * box_bytes * 2 * NS);
        __syncwarp();
        if (mine)
          tma_load_page(sa(ring + size_t(s) * C::kStage + slab * C::kSlab) + b * box_bytes, slab < NS ? &mk : &mv,
                        sa(&full[s]), (slab < NS ? slab : slab - NS) * 64, (key0 + b * box) & (page - 1), g.h, pid);
      }
    }
    // the copies in flight land before the CTA leaves
    for (int j = max(it - C::kStages, 0); j < it; ++j)
      bar_wait(&full[j % C::kStages], uint32_t(j / C::kStages) & 1u, err, ok ? kSpinCycles : kSpinCyclesAfterError);
    return;
  }

  // ---- compute warps
  const float sl = a.scale * 1.4426950408889634f;  // scores in powers of two
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  bool ok = true;
  while (walk.next(a, g)) {  // after a wait that gave up too: the warps meet at barriers
    const int tok0 = g.u * ut, n_tok = min(ut, g.q.q_len - tok0), n_rows = n_tok * a.group;
    int lim[2], lo[2];
    uint32_t q[4 * NS][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = r0 + 8 * i, tok = row / a.group;
      const bool there = row < n_rows;
      lim[i] = there ? attn_lim(a, g.q, tok0 + tok) : 0;
      lo[i] = attn_lo(a, lim[i]);
      const uint16_t* src = static_cast<const uint16_t*>(a.Q) + int64_t(g.q.q0 + tok0 + tok) * a.q_stride +
                            int64_t(g.h * a.group + row - tok * a.group) * a.dim;
#pragma unroll
      for (int k = 0; k < 4 * NS; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int c = k * 16 + x * 8 + c0;
          q[k][2 * x + i] = there && c < a.dim ? __ldcg(reinterpret_cast<const uint32_t*>(src + c)) : 0u;
        }
    }
    const int lim_all = attn_lim(a, g.q, tok0 + n_tok - 1), lim_min = attn_lim(a, g.q, tok0);  // last and first token's
    const int lo_all = attn_lo(a, lim_min), lo_max = attn_lo(a, lim_all);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[8 * NS][4];
#pragma unroll
    for (int n = 0; n < 8 * NS; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
    bool found = false;

    for (int i = g.a; i < g.b; ++i, ++it) {
      const int s = it % C::kStages;
      const int tile = (g.t0 + i) * kRowsKt;
      const bool partial = tile < lo_max || tile + kRowsKt > lim_min;
      ok = ok && __all_sync(0xffffffffu, bar_wait(&full[s], uint32_t(it / C::kStages) & 1u, err));
      if (!ok) continue;
      const uint32_t kb = sa(ring + size_t(s) * C::kStage), vb = kb + NS * C::kSlab;
      // scores of this warp's 16 keys: lane l addresses row l % 8 (+ 8 in lanes 16..31) of the fragment
      float sc[2][4] = {};
      {
        const int kr = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
        const uint32_t base = kb + kr * 128;
        const int ch = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 4 * NS; ++k) {
          uint32_t b[4];
          rows_ldsm(base + (k >> 2) * C::kSlab + ((((k & 3) * 2 + ch) ^ (kr & 7)) << 4), b);
          rows_mma(sc[0], q[k], b[0], b[1]);
          rows_mma(sc[1], q[k], b[2], b[3]);
        }
      }
      const int j0 = tile + warp * 16 + c0;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          sc[x][y] *= sl;
          if (partial) {
            const int j = j0 + 8 * x + (y & 1);
            if (j < lo[y >> 1] || j >= lim[y >> 1]) sc[x][y] = -INFINITY;
          }
        }
      float f[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float mx = fmaxf(fmaxf(sc[0][2 * y], sc[0][2 * y + 1]), fmaxf(sc[1][2 * y], sc[1][2 * y + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = fmaxf(mx, m[y]);
        f[y] = attn_scale(m[y], mx);
        m[y] = mx;
        const float to = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            sc[x][2 * y + z] = ex2(sc[x][2 * y + z] - to);
            sum += sc[x][2 * y + z];
          }
        l[y] = l[y] * f[y] + sum;  // this lane's keys; the lanes of a row are added at the end
      }
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int n = 0; n < 8 * NS; ++n) {
          o[n][0] *= f[0];
          o[n][1] *= f[0];
          o[n][2] *= f[1];
          o[n][3] *= f[1];
        }
      }
      // the weights enter the second product as bf16: 2^-9 of each, what their own rounding to the cache's type costs
      const uint32_t p[4] = {attn_pack(sc[0][0], sc[0][1]), attn_pack(sc[0][2], sc[0][3]), attn_pack(sc[1][0], sc[1][1]),
                             attn_pack(sc[1][2], sc[1][3])};
      {
        const int vr = warp * 16 + (lane & 15);
        const uint32_t base = vb + vr * 128;
#pragma unroll
        for (int n = 0; n < 4 * NS; ++n) {
          uint32_t b[4];
          rows_ldsm_t(base + (n >> 2) * C::kSlab + ((((n & 3) * 2 + (lane >> 4)) ^ (vr & 7)) << 4), b);
          if (partial) {
#pragma unroll
            for (int x = 0; x < 4; ++x) b[x] = rows_clean(b[x], j0 + 8 * (x & 1), lo_all, lim_all, found);
          }
          rows_mma(o[2 * n], p, b[0], b[1]);
          rows_mma(o[2 * n + 1], p, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&empty[s]);
    }

    // ---- the four warps' parts of the segment: common maximum, one sum
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
      if ((lane & 3) == 0) {
        s_ml[warp * 32 + r0 + 8 * y] = m[y];
        s_ml[warp * 32 + 16 + r0 + 8 * y] = l[y];
      }
    }
    if (found) s_flag[1] = 1;
    rows_sync();
    const bool any = s_flag[1] != 0;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float mx = s_ml[r0 + 8 * y];
#pragma unroll
      for (int w = 1; w < kRowsWarps; ++w) mx = fmaxf(mx, s_ml[w * 32 + r0 + 8 * y]);
      m[y] = attn_scale(m[y], mx);  // this warp's factor
    }
    for (int w = 0; w < kRowsWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (r0 + 8 * y < n_rows) {
#pragma unroll
            for (int n = 0; n < 8 * NS; ++n) {
              float2* dst = reinterpret_cast<float2*>(s_o + (r0 + 8 * y) * C::kDim + n * 8 + c0);
              float2 v = make_float2(o[n][2 * y] * m[y], o[n][2 * y + 1] * m[y]);
              if (w > 0) {
                const float2 u = *dst;
                v.x += u.x;
                v.y += u.y;
              }
              *dst = v;
            }
          }
      }
      rows_sync();
    }
    const bool whole = g.a == 0 && g.b == g.n;
    int b0, b1;
    walk.parts(g, b0, b1);
    float* part = attn_part(a, 2 * int(blockIdx.x) + (int(blockIdx.x) == b0), 1, 0, 16);
    const int vec = a.dim / 8;
    for (int e = tid; e < n_rows * vec; e += kRowsWarps * 32) {
      const int row = e / vec, c = (e - row * vec) * 8;
      float mx = s_ml[row], sum = 0.f;
#pragma unroll
      for (int w = 1; w < kRowsWarps; ++w) mx = fmaxf(mx, s_ml[w * 32 + row]);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) sum += s_ml[w * 32 + 16 + row] * attn_scale(s_ml[w * 32 + row], mx);
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = s_o[row * C::kDim + c + x];
      if (any) {
        const int rl = attn_lim(a, g.q, tok0 + row / a.group);
        for (int x = 0; x < 8; ++x)
          v[x] = attn_nonfinite<BF16>(a, g, kRowsKt, attn_lo(a, rl), rl, lo_max, lim_min, c + x, v[x]);
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] *= inv;
        attn_store8<BF16>(a, attn_out_row(a, g, tok0, row) * a.dim + c, v);
      } else {
        *attn_piece<true>(part, 16, a.dim, row, c) = make_float4(v[0], v[1], v[2], v[3]);
        *attn_piece<true>(part, 16, a.dim, row, c + 4) = make_float4(v[4], v[5], v[6], v[7]);
        if (c == 0) {
          part[row] = mx;
          part[16 + row] = sum;
        }
      }
    }
    if (!whole) {
      __threadfence();
      rows_sync();
      if (tid == 0) {
        const unsigned n = unsigned(b1 - b0 + 1);
        const bool last = atomicAdd(attn_counter(a, b0, 0), 1u) == n - 1;
        if (last) *attn_counter(a, b0, 0) = 0;
        s_flag[0] = last;
      }
      rows_sync();
      if (s_flag[0]) {
        __threadfence();
        attn_join<BF16, true, 8>(a, g, b0, b1, 1, 0, 16, n_rows, tok0, tid, kRowsWarps * 32);
      }
    }
    if (tid == 0) s_flag[1] = 0;
    rows_sync();  // before the next segment writes the shared rows
  }
}

template <int NS>
static cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  using C = RowsCfg<NS>;
  static_assert(C::kSmem <= 232448, "shared memory of an SM");
  const int box = (1 << a.page_shift) < kRowsKt ? (1 << a.page_shift) : kRowsKt;
  CUtensorMap mk, mv;
  cudaError_t e = attn_page_map(&mk, a, a.K, box);
  if (e == cudaSuccess) e = attn_page_map(&mv, a, a.V, box);
  if (e != cudaSuccess) return e;
  static bool set = false;  // a function attribute, the same for every call
  if (!set) {
    e = cudaFuncSetAttribute(attn_rows16_kernel<NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
    if (e != cudaSuccess) return e;
    set = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(min(attn_sm_count(), kAttnCtas));
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_rows16_kernel<NS>, mk, mv, a);
}

cudaError_t launch_attn_rows16(const AttnArgs& a, cudaStream_t s) {
  switch ((a.dim + 63) / 64) {
    case 1: return launch_rows<1>(a, s);
    case 2: return launch_rows<2>(a, s);
    case 3: return launch_rows<3>(a, s);
    default: return launch_rows<4>(a, s);
  }
}

}  // namespace gsi
