// Attention of few query rows (decode): a unit's at most 8 rows in one
// tensor-core tile, the keys and values streamed once.

#include "gsi_attn.cuh"

namespace gsi {

// With G = group query heads a key/value head and ut = floor(8 / G) tokens a
// unit, S = Q K^T and O = P V have at most 8 rows: 8 FLOP a byte of cache, far
// below what the warp-level tensor products sustain, so the bytes bound the
// kernel and its work is to keep them coming (16 requests of up to 8191 keys, 40
// x 128: 247 us, 6.2 TB/s; 260001 keys of 8 x 128: 165 us, 6.45 TB/s).  More
// rows go to the row tiles: a form of this kernel with all 16 rows of a fragment
// was slower than they are from 2000 keys on (19 against 16 us for 16 heads that
// share one of 8 key/value heads, 53 against 45 us at 8 x 8000 keys).  One CTA an SM;
// copy warps keep a ring of 192 KB filled (64 or 128 keys and their values a stage,
// one TMA box a page and 64 columns, each lane issuing its own box); eight warps
// take every stage, one to each 16 keys with a softmax of its own (running
// maximum m, sum l).  A stage's chain of products, maxima, exponentials and
// products has to be shorter than its 64 KB take to arrive (~2700 cycles): 128
// keys a stage up to 128 columns; above, 64 keys, and two warps to each 16 of
// them, which both form the scores and each half of the output's columns.  The
// warps' parts are joined when the CTA's part of a unit ends.  The scores'
// fragment of m16n8k16 is the next product's left operand as it stands, so P
// never leaves the registers.
template <int NS>  // 64-column slabs of a row
struct RowsCfg {
  static constexpr int kWarps = 8;                       // compute warps
  static constexpr int kKeyWarps = NS <= 2 ? 8 : 4;      // 16 keys of a stage each
  static constexpr int kColWarps = kWarps / kKeyWarps;   // with the same keys: parts of the columns
  static constexpr int kKt = 16 * kKeyWarps;             // keys a stage
  // three warpgroups: the copy warps' hands registers to the others
  static constexpr int kThreads = 384;
  static constexpr int kRows = 8, kShared = 16;          // query rows; output rows in shared memory
  static constexpr int kSlab = kKt * 128;                // bytes
  static constexpr int kStage = 2 * NS * kSlab;          // K slabs, then V slabs
  static constexpr int kStages = 196608 / kStage;        // 192 KB
  static constexpr int kDim = NS * 64;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + kShared * kDim * 4 + kKeyWarps * 16 * 4 + 2 * kStages * 8 + 16;
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
// c += a b, the upper 8 rows of the 16 (the lower ones are zeros that go nowhere).
__device__ __forceinline__ void rows_mma(float (&c)[2], const uint32_t (&a)[2], uint32_t b0, uint32_t b1) {
  float x = 0.f, y = 0.f;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %8, %5, %8}, {%6, %7}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(x), "+f"(y)
      : "r"(a[0]), "r"(a[1]), "r"(b0), "r"(b1), "r"(0u));
}
// The compute warps only.
template <int N>
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }

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
__global__ void __launch_bounds__(RowsCfg<NS>::kThreads, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                     const __grid_constant__ AttnArgs a) {
  using C = RowsCfg<NS>;
  constexpr int NW = C::kWarps;
  constexpr int KW = C::kKeyWarps, NO = 8 * NS / C::kColWarps;  // 8-column pieces of the output a warp holds
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_o = reinterpret_cast<float*>(ring + size_t(C::kStages) * C::kStage);  // [16][kDim]
  float* s_ml = s_o + C::kShared * C::kDim;                                      // [keys' warp][m: 8, l: 8]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ml + KW * 16);
  uint64_t* empty = full + C::kStages;
  int* s_flag = reinterpret_cast<int*>(empty + C::kStages);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      bar_init(&full[s], 4);
      bar_init(&empty[s], NW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mk) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mv) : "memory");
    s_flag[1] = 0;
  }
  pdl_wait();
  AttnWalk walk;
  const int ut = walk.ut = C::kRows / a.group;
  walk.kt = C::kKt;
  walk.s = attn_share<C::kThreads>(a, ut, C::kKt, 0, walk.p);  // also publishes the barriers to the block
  uint32_t* err = attn_err(a);
  AttnSeg g;
  int it = 0;  // stages so far

  if (warp >= NW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---- copy warps: a stage's boxes (at most 32: 2 NS slabs, a box a page) are dealt out to their lanes.  Four warps, because a
    // warp issues its lanes' boxes one after the other, ~80 cycles each: 16 of them take one warp as long as the
    // stage's bytes take to arrive.
    const int page = 1 << a.page_shift;
    const int box = min(page, C::kKt), boxes = C::kKt / box;  // tokens of a box; boxes of a slab
    const uint32_t box_bytes = uint32_t(box) * 128;
    bool ok = true;
    while (ok && walk.next(a, g)) {
      const int lim_all = attn_lim(a, g.q, min((g.u + 1) * ut, g.q.q_len) - 1);
      const int lo_all = attn_lo(a, attn_lim(a, g.q, g.u * ut));
      const int32_t* row = a.table + int64_t(g.r) * a.width;
      // this lane's box: slabs of K, then of V
      const int mine_no = lane * 4 + warp - NW, b = mine_no % boxes, slab = mine_no / boxes;
      // its page in tile i, if it has a key that some row sees (loaded a stage ahead: the table's latency is half a
      // stage's time)
      auto wanted = [&](int i) {
        const int key0 = (g.t0 + i) * C::kKt, first = max(lo_all - key0, 0) / box;
        return i < g.b && slab < 2 * NS && b >= first && key0 + b * box < lim_all;
      };
      auto page_of = [&](int i) { return wanted(i) ? __ldcg(row + (((g.t0 + i) * C::kKt + b * box) >> a.page_shift)) : 0; };
      int next = page_of(g.a);
      for (int i = g.a; i < g.b; ++i, ++it) {
        const int s = it % C::kStages;
        const int key0 = (g.t0 + i) * C::kKt;
        const bool mine = wanted(i);
        const int pid = next;
        next = page_of(i + 1);
        if (it >= C::kStages)
          ok = __all_sync(0xffffffffu, bar_wait(&empty[s], uint32_t(it / C::kStages - 1) & 1u, err));
        if (!ok) break;
        // each copy warp arrives for its own boxes, with none of them too: no warp falls behind a stage's next use
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) bar_expect_tx(&full[s], uint32_t(n) * box_bytes);
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

  // ---- compute warps: 16 keys of every stage (kg), and a part of the columns (dh)
  asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  const int kg = warp % KW, dh = warp / KW;
  const float sl = a.scale * 1.4426950408889634f;  // scores in powers of two
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  bool ok = true;
  while (walk.next(a, g)) {  // after a wait that gave up too: the warps meet at barriers
    const int tok0 = g.u * ut, n_tok = min(ut, g.q.q_len - tok0), n_rows = n_tok * a.group;
    uint32_t q[4 * NS][2];
    const int tok = r0 / a.group;
    const bool there = r0 < n_rows;
    const int lim = there ? attn_lim(a, g.q, tok0 + tok) : 0, lo = attn_lo(a, lim);
    const uint16_t* src = static_cast<const uint16_t*>(a.Q) + int64_t(g.q.q0 + tok0 + tok) * a.q_stride +
                          int64_t(g.h * a.group + r0 - tok * a.group) * a.dim;
#pragma unroll
    for (int k = 0; k < 4 * NS; ++k)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = k * 16 + x * 8 + c0;
        q[k][x] = there && c < a.dim ? __ldcg(reinterpret_cast<const uint32_t*>(src + c)) : 0u;
      }
    const int lim_all = attn_lim(a, g.q, tok0 + n_tok - 1), lim_min = attn_lim(a, g.q, tok0);  // last and first token's
    const int lo_all = attn_lo(a, lim_min), lo_max = attn_lo(a, lim_all);
    float m = -INFINITY, l = 0.f;
    float o[NO][2];
#pragma unroll
    for (int n = 0; n < NO; ++n) o[n][0] = o[n][1] = 0.f;
    bool found = false;

    for (int i = g.a; i < g.b; ++i, ++it) {
      const int s = it % C::kStages;
      const int tile = (g.t0 + i) * C::kKt;
      const bool partial = tile < lo_max || tile + C::kKt > lim_min;
      ok = ok && __all_sync(0xffffffffu, bar_wait(&full[s], uint32_t(it / C::kStages) & 1u, err));
      if (!ok) continue;
      const uint32_t kb = sa(ring + size_t(s) * C::kStage), vb = kb + NS * C::kSlab;
      // scores of this warp's 16 keys, in two chains of products; lane l addresses row l % 8 (+ 8 in lanes 16..31) of
      // the fragment
      float sc[2][2];
      {
        float part[2][2][2] = {};
        const int kr = kg * 16 + (lane & 7) + ((lane >> 4) << 3);
        const uint32_t base = kb + kr * 128;
        const int ch = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 4 * NS; ++k) {
          uint32_t b[4];
          rows_ldsm(base + (k >> 2) * C::kSlab + ((((k & 3) * 2 + ch) ^ (kr & 7)) << 4), b);
          rows_mma(part[k & 1][0], q[k], b[0], b[1]);
          rows_mma(part[k & 1][1], q[k], b[2], b[3]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) sc[x][y] = (part[0][x][y] + part[1][x][y]) * sl;
      }
      const int j0 = tile + kg * 16 + c0;
      if (partial) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int j = j0 + 8 * x + y;
            if (j < lo || j >= lim) sc[x][y] = -INFINITY;
          }
      }
      float mx = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      mx = fmaxf(mx, m);
      const float f = attn_scale(m, mx), to = mx == -INFINITY ? 0.f : mx;
      m = mx;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) sc[x][y] = ex2(sc[x][y] - to);
      // the weights enter the second product as bf16: 2^-8 of each at most, what rounding to the cache's type costs; what
      // enters it is what is summed, so that the output is a mean of the values for any rounding
      const uint32_t p[2] = {attn_pack(sc[0][0], sc[0][1]), attn_pack(sc[1][0], sc[1][1])};
#pragma unroll
      for (int x = 0; x < 2; ++x) BF16::unpack2(p[x], sc[x][0], sc[x][1]);
      l = l * f + ((sc[0][0] + sc[0][1]) + (sc[1][0] + sc[1][1]));  // this lane's keys; the lanes of a row are added at the end
      if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          o[n][0] *= f;
          o[n][1] *= f;
        }
      }
      {
        const int vr = kg * 16 + (lane & 15);
        const uint32_t base = vb + vr * 128;
#pragma unroll
        for (int n = 0; n < NO / 2; ++n) {
          const int c16 = dh * (NO / 2) + n;  // 16 columns
          uint32_t b[4];
          rows_ldsm_t(base + (c16 >> 2) * C::kSlab + ((((c16 & 3) * 2 + (lane >> 4)) ^ (vr & 7)) << 4), b);
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

    // ---- the warps' parts of the segment: common maximum, one sum.  The shared rows hold 16 / n_rows copies of the
    // output; in each round the warps of that many 16 keys add to a copy each, in their order, and the
    // copies are added at the end.
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (dh == 0 && (lane & 3) == 0) {
      s_ml[kg * 16 + r0] = m;
      s_ml[kg * 16 + 8 + r0] = l;
    }
    if (found) s_flag[1] = 1;
    rows_sync<NW * 32>();
    const bool any = s_flag[1] != 0;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < KW; ++w) mx = fmaxf(mx, s_ml[w * 16 + r0]);
    const float mine = attn_scale(m, mx);  // this warp's factor
    const int copies = min(KW, C::kShared / n_rows), rounds = (KW + copies - 1) / copies;
    for (int round = 0; round < rounds; ++round) {
      if (kg / copies == round && r0 < n_rows) {
        float* row = s_o + ((kg % copies) * n_rows + r0) * C::kDim + dh * (NO * 8);
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          float2* dst = reinterpret_cast<float2*>(row + n * 8 + c0);
          float2 v = make_float2(o[n][0] * mine, o[n][1] * mine);
          if (round > 0) {
            const float2 u = *dst;
            v.x += u.x;
            v.y += u.y;
          }
          *dst = v;
        }
      }
      rows_sync<NW * 32>();
    }
    const bool whole = g.a == 0 && g.b == g.n;
    int b0, b1;
    walk.parts(g, b0, b1);
    float* part = attn_part(a, 2 * int(blockIdx.x) + (int(blockIdx.x) == b0), 1, 0, C::kRows);
    const int vec = a.dim / 8;
    for (int e = tid; e < n_rows * vec; e += NW * 32) {
      const int row = e / vec, c = (e - row * vec) * 8;
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) mx = fmaxf(mx, s_ml[w * 16 + row]);
#pragma unroll
      for (int w = 0; w < KW; ++w) sum += s_ml[w * 16 + 8 + row] * attn_scale(s_ml[w * 16 + row], mx);
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = s_o[row * C::kDim + c + x];
      for (int k = 1; k < copies; ++k)
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] += s_o[(k * n_rows + row) * C::kDim + c + x];
      if (any) {
        const int rl = attn_lim(a, g.q, tok0 + row / a.group);
        for (int x = 0; x < 8; ++x)
          v[x] = attn_nonfinite<BF16>(a, g, C::kKt, attn_lo(a, rl), rl, lo_max, lim_min, c + x, v[x]);
      }
      if (whole) {
        attn_finish<BF16, 8>(a, g.q, tok0 + row / a.group, attn_out_row(a, g, tok0, row) * a.dim + c, c, sum, v);
      } else {
        *attn_piece<true>(part, C::kRows, a.dim, row, c) = make_float4(v[0], v[1], v[2], v[3]);
        *attn_piece<true>(part, C::kRows, a.dim, row, c + 4) = make_float4(v[4], v[5], v[6], v[7]);
        if (c == 0) {
          part[row] = mx;
          part[C::kRows + row] = sum;
        }
      }
    }
    if (!whole) {
      __threadfence();
      rows_sync<NW * 32>();
      if (tid == 0) {
        const unsigned n = unsigned(b1 - b0 + 1);
        const bool last = atomicAdd(attn_counter(a, b0, 0), 1u) == n - 1;
        if (last) *attn_counter(a, b0, 0) = 0;
        s_flag[0] = last;
      }
      rows_sync<NW * 32>();
      if (s_flag[0]) {
        __threadfence();
        attn_join<BF16, true, 8>(a, g, b0, b1, 1, 0, C::kRows, n_rows, tok0, tid, NW * 32);
      }
    }
    if (tid == 0) s_flag[1] = 0;
    rows_sync<NW * 32>();  // before the next segment writes the shared rows
  }
}

template <int NS>
static cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  using C = RowsCfg<NS>;
  static_assert(C::kSmem + 512 <= 232448, "shared memory of an SM, some of it static");
  const int box = (1 << a.page_shift) < C::kKt ? (1 << a.page_shift) : C::kKt;
  CUtensorMap mk, mv;
  cudaError_t e = attn_page_map(&mk, a, a.K, box);
  if (e == cudaSuccess) e = attn_page_map(&mv, a, a.V, box);
  if (e != cudaSuccess) return e;
  static OnEveryDevice ready;
  e = ready([] { return attn_prepare_kernel(attn_rows_kernel<NS>, C::kSmem, C::kThreads, 72 * 128 + 216 * 256); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(min(sm_count(), kAttnCtas));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_rows_kernel<NS>, mk, mv, a);
}

cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t s) {
  switch ((a.dim + 63) / 64) {
    case 1: return launch_rows<1>(a, s);
    case 2: return launch_rows<2>(a, s);
    case 3: return launch_rows<3>(a, s);
    default: return launch_rows<4>(a, s);
  }
}

}  // namespace gsi
