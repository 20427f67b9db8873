// Accumulated attention weights of the keys of a bf16 cache, on the tensor cores
// (tcgen05, TMEM), sm_103a.

#include "gsi_attn.cuh"
#include "gsi_tcgen.cuh"
#include "gsi_weights.cuh"

namespace gsi {

// A unit is 128 keys, a step up to NR query rows: S^T = K Q^T with the keys along
// the 128 lanes of TMEM, so that a thread owns a key and its sum over the rows
// needs no exchange.  Roles: one thread issues the products; two warps copy K, a
// box a page and 64 columns; one warp copies the steps' rows of Q and hands their
// logarithms over in shared memory; two warpgroups take the steps in turn
// (score, scaling and logarithm in one fused product, an exponential, a sum) and
// add their halves when the unit ends.
//   NR = 16: few rows (single tokens).  A unit is a step as a rule, and the bytes
//            of K bound it: a ring of 200 KB keeps them coming;
//   NR = 128: many.  K stays while the rows pass; the exponentials bound it (one
//            a pair, 16 a cycle and SM), above 128 columns the products.
constexpr int kKtKeys = 128, kKtSlab = 16384;  // 64 columns of 128 keys

template <int NS, int NR>
struct KtCfg {
  static constexpr int kKBytes = NS * kKtSlab, kQBytes = NS * NR * 128;
  static constexpr int kKBufs = NR == 16 ? 221184 / (kKBytes + kQBytes) : NS <= 2 ? 2 : 1;
  static constexpr int kQBufs = NR == 16 ? kKBufs : (221184 - kKBufs * kKBytes) / kQBytes < 6 ? (221184 - kKBufs * kKBytes) / kQBytes : 6;
  static constexpr int kSBufs = NR == 16 ? 8 : 4;  // accumulators in TMEM
  static constexpr int kCols = kSBufs * NR;
  static constexpr int kSumWarps = 8, kThreads = 32 * (kSumWarps + 4);
  static constexpr size_t kSmem = 1024 + size_t(kKBufs) * kKBytes + size_t(kQBufs) * kQBytes + kSBufs * NR * 4 + 2 * 128 * 4 + 1024;
  static_assert(kSmem <= 232448 - 1024 && kKBufs <= 12 && kQBufs <= 12, "shared memory of an SM, some of it static");
  static_assert(kCols == 128 || kCols == 512, "TMEM is had in powers of two");
};

struct KtBars {
  uint64_t k_full[12], k_empty[12], q_full[12], q_empty[12];
  uint64_t s_full[8], s_empty[8], lse_full[8];
  uint64_t done;
  uint32_t tmem;
  int last[2];
};
static_assert(sizeof(KtBars) <= 1024, "barriers");

// 16 columns of this warp's 32 lanes (no wait).
__device__ __forceinline__ void kt_ld16(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : GSI_R8(r, 0), GSI_R8(r, 8)
               : "r"(t));
}
__device__ __forceinline__ void kt_arrived16(uint32_t* r) { asm volatile("" : GSI_H8(r, 0), GSI_H8(r, 8)::"memory"); }

template <int NS, int NR>
__global__ void __launch_bounds__(KtCfg<NS, NR>::kThreads, 1)
    key_weights_tiles_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                             const __grid_constant__ KeyWeightArgs a, int tpt) {
  using C = KtCfg<NS, NR>;
  constexpr int KB = C::kKBufs, QB = C::kQBufs, SB = C::kSBufs;
  extern __shared__ uint8_t kt_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kt_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* s_k = base;
  uint8_t* s_q = s_k + KB * C::kKBytes;
  float* s_lse = reinterpret_cast<float*>(s_q + QB * C::kQBytes);  // [SB][NR], negated
  float* s_half = s_lse + SB * NR;                                 // [2][128]
  KtBars& bars = *reinterpret_cast<KtBars*>(s_half + 2 * 128);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < KB; ++i) {
      bar_init(&bars.k_full[i], 2);
      bar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < QB; ++i) {
      bar_init(&bars.q_full[i], 1);
      bar_init(&bars.q_empty[i], 1);
    }
    for (int i = 0; i < SB; ++i) {
      bar_init(&bars.s_full[i], 1);
      bar_init(&bars.s_empty[i], 4);
      bar_init(&bars.lse_full[i], 1);
    }
    bar_init(&bars.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mq) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mk) : "memory");
  }
  if (warp == C::kSumWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&bars.tmem)), "r"(uint32_t(C::kCols)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tl_fence_before();
  pdl_wait();
  KwWalk<kKtKeys> walk;
  kw_share<kKtKeys, C::kThreads>(a, tpt, walk);  // its block barriers publish the ones above
  tl_fence_after();
  const uint32_t tmem = bars.tmem;
  uint32_t* err = kw_err(a);
  KwSeg g;
  bool ok = true;
  const int box_rows = tpt * a.group;  // of Q's boxes

  if (warp == C::kSumWarps) {
    // ---- the products (one thread)
    if (tl_elect()) {
      const uint64_t dk = tl_desc(sa(s_k), 0), dq = tl_desc(sa(s_q), 0);
      const uint32_t id = tl_idesc((box_rows + 15) / 16 * 16, false);
      int kb = 0, qb = 0, sb = 0;
      uint32_t kp = 0, qp = 0, sp = 1;  // the first wait for a free accumulator passes
      while (ok && walk.next(a, g)) {
        if (g.q.q_len == 0) continue;
        ok = bar_wait(&bars.k_full[kb], kp, err);
        for (int i = g.a; ok && i < g.b; ++i) {
          ok = bar_wait(&bars.q_full[qb], qp, err) && bar_wait(&bars.s_empty[sb], sp, err);
          if (!ok) break;
          tl_fence_after();
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const uint64_t ad = dk + uint64_t(kb * C::kKBytes + s * kKtSlab) / 16;
            const uint64_t bd = dq + uint64_t(qb * C::kQBytes + s * NR * 128) / 16;
#pragma unroll
            for (int k = 0; k < 4; ++k) tl_mma_ss(tmem + sb * NR, ad + uint64_t(2 * k), bd + uint64_t(2 * k), id, (s | k) != 0);
          }
          tl_commit(&bars.s_full[sb]);
          tl_commit(&bars.q_empty[qb]);
          if (++qb == QB) qb = 0, qp ^= 1;
          if (++sb == SB) sb = 0, sp ^= 1;
        }
        if (!ok) break;
        tl_commit(&bars.k_empty[kb]);
        if (++kb == KB) kb = 0, kp ^= 1;
      }
      tl_commit(&bars.done);
      bar_wait(&bars.done, 0, err, ok ? kSpinCycles : kSpinCyclesAfterError);
    }
    __syncwarp();
  } else if (warp == C::kSumWarps + 1) {
    // ---- rows of Q, and their logarithms
    int qb = 0, sb = 0, used = 0;
    uint32_t qp = 1, sp = 1;
    while (ok && walk.next(a, g)) {
      if (g.q.q_len == 0) continue;
      for (int i = g.a; ok && i < g.b; ++i) {
        const int tok0 = (g.u0 + i) * tpt;
        const int n_rows = min(tpt, g.q.q_len - tok0) * a.group;
        float l[NR == 16 ? 1 : 4];
        constexpr int NL = NR == 16 ? 1 : 4;
#pragma unroll
        for (int x = 0; x < NL; ++x) {
          const int row = lane + 32 * x, tok = row / a.group;
          l[x] = row < n_rows ? __ldcg(a.LSE + (int64_t(g.q.q0 + tok0 + tok) * a.hkv + g.h) * a.group + (row - tok * a.group)) : 0.f;
        }
        ok = __all_sync(0xffffffffu, bar_wait(&bars.q_empty[qb], qp, err));
        if (!ok) break;
        if (lane == 0) bar_expect_tx(&bars.q_full[qb], uint32_t(NS * box_rows) * 128);
        __syncwarp();
        if (lane < NS)
          tl_load_query(sa(s_q + qb * C::kQBytes + lane * NR * 128), &mq, sa(&bars.q_full[qb]), lane * 64, g.h * a.group, g.q.q0 + tok0);
        used = min(used + 1, QB);
        if (++qb == QB) qb = 0, qp ^= 1;
        ok = __all_sync(0xffffffffu, bar_wait(&bars.s_empty[sb], sp, err));
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < NL; ++x)
          if (lane + 32 * x < NR) s_lse[sb * NR + lane + 32 * x] = -l[x];
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.lse_full[sb]);
        if (++sb == SB) sb = 0, sp ^= 1;
      }
    }
    // the copies in flight land before the CTA leaves: the last use of every buffer that was filled
    for (int i = 0; i < used; ++i) {
      const int s = qb - 1 - i;
      bar_wait(&bars.q_full[s < 0 ? s + QB : s], s < 0 ? qp : qp ^ 1u, err, ok ? kSpinCycles : kSpinCyclesAfterError);
    }
  } else if (warp >= C::kSumWarps + 2) {
    // ---- keys: two warps share a tile's boxes
    const int page = 1 << a.page_shift, box = min(page, kKtKeys), boxes = kKtKeys / box;
    const int no = lane * 2 + warp - (C::kSumWarps + 2), b = no % boxes, slab = no / boxes;
    int kb = 0, used = 0;
    uint32_t kp = 1;
    while (ok && walk.next(a, g)) {
      if (g.q.q_len == 0) continue;
      const int key0 = g.t * kKtKeys, key = key0 + b * box;
      const bool mine = slab < NS && key < g.q.len;
      const int pid = mine ? __ldcg(a.table + int64_t(g.r) * a.width + (key >> a.page_shift)) : 0;
      ok = __all_sync(0xffffffffu, bar_wait(&bars.k_empty[kb], kp, err));
      if (!ok) break;
      const int n = __popc(__ballot_sync(0xffffffffu, mine));
      if (lane == 0) bar_expect_tx(&bars.k_full[kb], uint32_t(n * box) * 128);
      __syncwarp();
      if (mine)
        tma_load_page(sa(s_k + kb * C::kKBytes + slab * kKtSlab) + b * box * 128, &mk, sa(&bars.k_full[kb]), slab * 64, key & (page - 1),
                      g.h, pid);
      used = min(used + 1, KB);
      if (++kb == KB) kb = 0, kp ^= 1;
    }
    for (int i = 0; i < used; ++i) {
      const int s = kb - 1 - i;
      bar_wait(&bars.k_full[s < 0 ? s + KB : s], s < 0 ? kp : kp ^ 1u, err, ok ? kSpinCycles : kSpinCyclesAfterError);
    }
  } else {
    // ---- sums: a thread a key, the two warpgroups take the steps in turn
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const float scale = a.scale;
    const unsigned long long c2 = f2_pack(scale, scale), e2 = f2_pack(1.4426950408889634f, 1.4426950408889634f);
    int step = 0, pair = 0;  // steps and units of several steps so far
    auto wg_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
    while (walk.next(a, g)) {  // after a wait that gave up too: the warps meet at barriers
      const int key = g.t * kKtKeys + row;
      const int n_steps = g.q.q_len > 0 ? g.b - g.a : 0;
      const int ends = n_steps > 0 ? (step + n_steps - 1) & 1 : 0;  // the warpgroup that ends the part
      const bool whole = g.a == 0 && g.b == g.n;
      KwMark mark{-1, 0.f, 0};
      if (whole && wg == ends) mark = kw_mark(a, g, key);  // ahead of the wait for the scores
      unsigned long long acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
      for (int i = 0; i < n_steps; ++i, ++step) {
        if ((step & 1) != wg) continue;
        const int sb = step % SB;
        const uint32_t ph = uint32_t(step / SB) & 1u;
        ok = ok && __all_sync(0xffffffffu, bar_wait(&bars.s_full[sb], ph, err) && bar_wait(&bars.lse_full[sb], ph, err));
        if (!ok) continue;
        tl_fence_after();
        const int tok0 = (g.u0 + g.a + i) * tpt;
        const int n_rows = min(tpt, g.q.q_len - tok0) * a.group;
        // the key is seen from this row of the step on
        const int late = a.causal ? min(max((key - g.q.len) + (g.q.q_len - tok0), 0), NR) * a.group : 0;
        const bool masked = __any_sync(0xffffffffu, late > 0);
        const float* lse = s_lse + sb * NR;
        constexpr int CH = NR == 16 ? 16 : 32;
#pragma unroll 1
        for (int c = 0; c < n_rows; c += CH) {
          uint32_t sr[CH];
          if constexpr (CH == 16) {
            kt_ld16(tmem + lanes + sb * NR + c, sr);
            tl_wait_ld();
            kt_arrived16(sr);
          } else {
            tl_ld32(tmem + lanes + sb * NR + c, sr);
            tl_wait_ld();
            tl_arrived32(sr);
          }
          const bool part = masked || c + CH > n_rows;
          uint32_t see = ~0u;
          if (part) {
            const int from = late - c, to = n_rows - c;
            const uint32_t below_to = to >= 32 ? ~0u : (1u << to) - 1u;
            see = from >= 32 ? 0u : from <= 0 ? below_to : below_to & ~((1u << from) - 1u);
          }
#pragma unroll
          for (int x = 0; x < CH; x += 4) {
            const float4 l = *reinterpret_cast<const float4*>(lse + c + x);
            float2 u = f2_unpack(f2_mul(f2_fma(f2_pack(__uint_as_float(sr[x]), __uint_as_float(sr[x + 1])), c2, f2_pack(l.x, l.y)), e2));
            float2 v = f2_unpack(f2_mul(f2_fma(f2_pack(__uint_as_float(sr[x + 2]), __uint_as_float(sr[x + 3])), c2, f2_pack(l.z, l.w)), e2));
            if (part) {
              if (!(see >> x & 1u)) u.x = -INFINITY;
              if (!(see >> (x + 1) & 1u)) u.y = -INFINITY;
              if (!(see >> (x + 2) & 1u)) v.x = -INFINITY;
              if (!(see >> (x + 3) & 1u)) v.y = -INFINITY;
            }
            acc[0] = f2_add(acc[0], f2_pack(ex2(u.x), ex2(u.y)));
            acc[1] = f2_add(acc[1], f2_pack(ex2(v.x), ex2(v.y)));
          }
        }
        tl_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.s_empty[sb]);
      }
      const float2 s01 = f2_unpack(f2_add(acc[0], acc[1]));
      float sum = s01.x + s01.y;
      if (n_steps > 1) {  // the other warpgroup's half
        float* half = s_half + (pair & 1) * 128;
        ++pair;
        if (wg != ends) half[row] = sum;
        asm volatile("bar.sync 3, 256;" ::: "memory");
        if (wg == ends) sum += half[row];
      }
      if (wg != ends) continue;
      if (whole) {
        kw_give(a, g, key, mark, sum);
        continue;
      }
      int b0, b1;
      walk.parts(g, b0, b1);
      kw_part(a, 2 * int(blockIdx.x) + (int(blockIdx.x) == b0))[row] = sum;
      __threadfence();
      wg_sync();
      if ((warp & 3) == 0 && lane == 0) {
        const bool last = atomicAdd(kw_counter(a, b0), 1u) == unsigned(b1 - b0);
        if (last) *kw_counter(a, b0) = 0;
        bars.last[wg] = last;
      }
      wg_sync();
      if (*reinterpret_cast<volatile int*>(&bars.last[wg])) {
        __threadfence();
        sum = 0.f;
        for (int b = b0; b <= b1; ++b) sum += __ldcg(kw_part(a, 2 * b + (b == b0)) + row);
        kw_give(a, g, key, kw_mark(a, g, key), sum);
      }
      wg_sync();  // before the flag is written again
    }
  }
  tl_fence_before();
  __syncthreads();
  if (warp == C::kSumWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(uint32_t(C::kCols)) : "memory");
}

template <int NS, int NR>
static cudaError_t launch_kt(const KeyWeightArgs& a, cudaStream_t s) {
  using C = KtCfg<NS, NR>;
  AttnArgs m{};  // what the maps are made of
  m.page_stride = a.page_stride;
  m.head_stride = a.head_stride;
  m.token_stride = a.token_stride;
  m.n_pages = a.n_pages;
  m.page_shift = a.page_shift;
  m.hkv = a.hkv;
  m.group = a.group;
  m.dim = a.dim;
  m.Q = a.Q;
  m.q_stride = a.q_stride;
  m.N = a.N;
  int tpt = 1;
  while (2 * tpt * a.group <= NR) tpt *= 2;
  const int page = 1 << a.page_shift;
  CUtensorMap mq, mk;
  cudaError_t e = attn_query_map(&mq, m, a.group, tpt);
  if (e == cudaSuccess) e = attn_page_map(&mk, m, a.K, page < kKtKeys ? page : kKtKeys);
  if (e != cudaSuccess) return e;
  static OnEveryDevice ready;
  e = ready([] { return attn_prepare_kernel(key_weights_tiles_kernel<NS, NR>, C::kSmem, C::kThreads, 0); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(min(sm_count(), kKwCtas));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_tiles_kernel<NS, NR>, mq, mk, a, tpt);
}

template <int NR>
static cudaError_t launch_kt_dim(const KeyWeightArgs& a, cudaStream_t s) {
  switch ((a.dim + 63) / 64) {
    case 1: return launch_kt<1, NR>(a, s);
    case 2: return launch_kt<2, NR>(a, s);
    case 3: return launch_kt<3, NR>(a, s);
    default: return launch_kt<4, NR>(a, s);
  }
}

cudaError_t launch_key_weights_tiles(const KeyWeightArgs& a, bool few, cudaStream_t s) {
  return few ? launch_kt_dim<16>(a, s) : launch_kt_dim<128>(a, s);
}

}  // namespace gsi
