// Accumulated attention weights of the keys of a bf16 cache, on the tensor cores
// (tcgen05, TMEM), sm_103a.

#include "gsi_attn.cuh"
#include "gsi_tcgen.cuh"
#include "gsi_weights.cuh"

namespace gsi {

// A unit is 128 keys, a step up to NR query rows: S^T = K Q^T with the keys along
// the 128 lanes of TMEM, so that a thread owns a key and its sum over the rows
// needs no exchange.  Roles: one thread issues the products; two or three warps
// copy K, a box a page and 64 columns; one warp copies the steps' rows of Q and
// hands their logarithms over in shared memory; two warpgroups take the steps in
// turn (score, scaling and logarithm in one fused product, an exponential, a sum)
// and add their halves where a unit has several.
//   NR = 16: few rows (single tokens).  A unit is a step as a rule, and the bytes
//            of K bound it: a ring of 200 KB keeps them coming, page numbers are
//            loaded several units ahead, and a warp brings what the keys have
//            gathered (a unit's ~700 ns do not hold the two loads, one behind the
//            other, that this takes a thread: 160 us with them, 143 without,
//            16 requests of 8191 keys, 40 x 128);
//   NR = 128: many.  K stays while the rows pass: 8192 tokens of 32/8 x 128 284 us,
//            of 32 x 64 292, of 16 x 256 197 (1.40 PFLOP/s).  A step takes ~1250 cycles at
//            64 and at 128 columns, ~1750 at 256; its exponentials take 512, its
//            products 4 a column: neither bounds it below 256 columns, nor do the
//            sums by themselves (~1400 a step and warpgroup, which has every
//            second step).  What does has not been found.  (256 keys over 64 rows a step, which
//            halves the reads of Q, was no faster while the rows' logarithms
//            bounded both: 27.0 against 24.3 us for 2048 tokens of 16 x 256, 235
//            against 229 for 8192; not tried again since they do not.)
constexpr int kKtSlab = 16384;                 // 64 columns of 128 keys

template <int NS, int NR>
struct KtCfg {
  static constexpr bool kFew = NR == 16;
  static constexpr int kKBytes = NS * kKtSlab, kQBytes = NS * NR * 128;
  static constexpr int kKBufs = kFew ? 221184 / (kKBytes + kQBytes) : NS <= 2 ? 2 : 1;
  static constexpr int kQRoom = (221184 - kKBufs * kKBytes) / kQBytes;
  static constexpr int kQBufs = kFew ? kKBufs : kQRoom < 6 ? kQRoom : 6;
  static constexpr int kSBufs = kFew ? 8 : 4;  // accumulators in TMEM
  static constexpr int kCols = kSBufs * NR;
  static constexpr int kMarks = kFew ? 8 : 0;  // units whose keys' weights are loaded ahead
  static constexpr int kAhead = kFew ? 3 : 1;  // items whose numbers are loaded ahead (each delays the first one)
  static constexpr int kSumWarps = 8, kCopyWarps = kFew ? 3 : 2, kThreads = 32 * (kSumWarps + 2 + kCopyWarps + (kFew ? 1 : 0));
  static constexpr size_t kSmem = 1024 + size_t(kKBufs) * kKBytes + size_t(kQBufs) * kQBytes + kSBufs * NR * 4 + 2 * 128 * 4 + kMarks * (128 * 4 + 128) + 1024;
  static_assert(kSmem <= 232448 - 1024 && kKBufs <= 12 && kQBufs <= 12, "shared memory of an SM, some of it static");
  static_assert(kCols == 128 || kCols == 512, "TMEM is had in powers of two");
};

struct KtBars {
  uint64_t k_full[12], k_empty[12], q_full[12], q_empty[12];
  uint64_t s_full[8], s_empty[8], lse_full[8];
  uint64_t mark_full[8], mark_empty[8];
  uint64_t done;
  uint32_t tmem;
  int last[2];
};
static_assert(sizeof(KtBars) <= 1024, "barriers");

// Items of a part, each with loads of its own that are issued D items before it is taken.
template <class T, int D>
struct KtAhead {
  T item[D];
  bool there[D];
  template <class F>
  __device__ __forceinline__ void start(F next) {
#pragma unroll
    for (int i = 0; i < D; ++i) there[i] = next(item[i]);
  }
  template <class F>
  __device__ __forceinline__ bool take(T& x, F next) {
    x = item[0];
    const bool some = there[0];
#pragma unroll
    for (int i = 0; i + 1 < D; ++i) {
      item[i] = item[i + 1];
      there[i] = there[i + 1];
    }
    there[D - 1] = there[D - 1] && next(item[D - 1]);
    return some;
  }
};

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
  constexpr int KB = C::kKBufs, QB = C::kQBufs, SB = C::kSBufs, KT = 128;
  extern __shared__ uint8_t kt_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kt_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* s_k = base;
  uint8_t* s_q = s_k + KB * C::kKBytes;
  float* s_lse = reinterpret_cast<float*>(s_q + QB * C::kQBytes);  // [SB][NR], negated
  float* s_half = s_lse + SB * NR;                                 // [2][128]
  float* s_old = s_half + 2 * 128;                                 // [kMarks][KT]: what a unit's keys have gathered
  int* s_page = reinterpret_cast<int*>(s_old + C::kMarks * KT);     // [kMarks][KT / 4]: the page of every fourth key
  KtBars& bars = *reinterpret_cast<KtBars*>(s_page + C::kMarks * KT / 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < KB; ++i) {
      bar_init(&bars.k_full[i], C::kCopyWarps);
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
    for (int i = 0; i < C::kMarks; ++i) {
      bar_init(&bars.mark_full[i], 33);
      bar_init(&bars.mark_empty[i], 8);
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
  KwWalk<KT> walk;
  kw_share<KT, C::kThreads>(a, tpt, walk);  // its block barriers publish the ones above
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
    // ---- rows of Q, and their logarithms (loaded three steps ahead: at one step ahead this chain was what bounded many
    // rows, ~1500 cycles a step where the sums take ~700)
    constexpr int NL = (NR + 31) / 32;
    struct Rows {
      int head, tok;  // of Q
      float l[NL];
    };
    int64_t off[NL];  // of this lane's rows in LSE
#pragma unroll
    for (int z = 0; z < NL; ++z) {
      const int row = lane + 32 * z, tok = row / a.group;
      off[z] = int64_t(tok) * a.hkv * a.group + (row - tok * a.group);
    }
    int i = 0, n = 0;  // steps of the part: this one, all
    bool have = false;
    auto next_rows = [&](Rows& x) {
      while (!have || i == n) {
        have = walk.next(a, g);
        if (!have) return false;
        i = g.a;
        n = g.q.q_len > 0 ? g.b : g.a;
      }
      const int tok0 = (g.u0 + i++) * tpt;
      const int n_rows = min(tpt, g.q.q_len - tok0) * a.group;
      x.head = g.h * a.group;
      x.tok = g.q.q0 + tok0;
      const float* from = a.LSE + int64_t(x.tok) * a.hkv * a.group + x.head;
#pragma unroll
      for (int z = 0; z < NL; ++z) x.l[z] = lane + 32 * z < n_rows ? __ldcg(from + off[z]) : 0.f;
      return true;
    };
    int qb = 0, sb = 0, used = 0;
    uint32_t qp = 1, sp = 1;
    KtAhead<Rows, 3> ahead;
    ahead.start(next_rows);
    Rows now;
    while (ok && ahead.take(now, next_rows)) {
      ok = __all_sync(0xffffffffu, bar_wait(&bars.q_empty[qb], qp, err));
      if (!ok) break;
      if (lane == 0) bar_expect_tx(&bars.q_full[qb], uint32_t(NS * box_rows) * 128);
      __syncwarp();
      if (lane < NS) tl_load_query(sa(s_q + qb * C::kQBytes + lane * NR * 128), &mq, sa(&bars.q_full[qb]), lane * 64, now.head, now.tok);
      used = min(used + 1, QB);
      if (++qb == QB) qb = 0, qp ^= 1;
      ok = __all_sync(0xffffffffu, bar_wait(&bars.s_empty[sb], sp, err));
      if (!ok) break;
#pragma unroll
      for (int z = 0; z < NL; ++z)
        if (lane + 32 * z < NR) s_lse[sb * NR + lane + 32 * z] = -now.l[z];
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.lse_full[sb]);
      if (++sb == SB) sb = 0, sp ^= 1;
    }
    // the copies in flight land before the CTA leaves: the last use of every buffer that was filled
    for (int i = 0; i < used; ++i) {
      const int s = qb - 1 - i;
      bar_wait(&bars.q_full[s < 0 ? s + QB : s], s < 0 ? qp : qp ^ 1u, err, ok ? kSpinCycles : kSpinCyclesAfterError);
    }
  } else if (warp >= C::kSumWarps + 2 && warp < C::kSumWarps + 2 + C::kCopyWarps) {
    // ---- keys: the warps share a tile's boxes (a warp issues its lanes' boxes one after the other, ~80 cycles each: 16
    // of them take one warp as long as the tile takes to arrive), each with the page numbers of the next tiles under way
    const int page = 1 << a.page_shift, box = min(page, 128), boxes = 128 / box;  // boxes of a slab
    const int no = lane * C::kCopyWarps + warp - (C::kSumWarps + 2), b = no % boxes, slab = no / boxes;
    struct Box {
      int tok, head, page;  // page: of the table
      bool mine;
    };
    auto next_box = [&](Box& x) {
      do {
        if (!walk.next(a, g)) return false;
      } while (g.q.q_len == 0);
      const int key = g.t * KT + b * box;
      x.mine = slab < NS && key < g.q.len;
      x.tok = key & (page - 1);
      x.head = g.h;
      x.page = x.mine ? __ldcg(a.table + int64_t(g.r) * a.width + (key >> a.page_shift)) : 0;
      return true;
    };
    int kb = 0, used = 0;
    uint32_t kp = 1;
    KtAhead<Box, C::kAhead> ahead;
    ahead.start(next_box);
    Box now;
    while (ok && ahead.take(now, next_box)) {
      ok = __all_sync(0xffffffffu, bar_wait(&bars.k_empty[kb], kp, err));
      if (!ok) break;
      const int n = __popc(__ballot_sync(0xffffffffu, now.mine));
      if (lane == 0) bar_expect_tx(&bars.k_full[kb], uint32_t(n * box) * 128);
      __syncwarp();
      if (now.mine)
        tma_load_page(sa(s_k + kb * C::kKBytes + slab * kKtSlab) + b * box * 128, &mk, sa(&bars.k_full[kb]), slab * 64, now.tok, now.head,
                      now.page);
      used = min(used + 1, KB);
      if (++kb == KB) kb = 0, kp ^= 1;
    }
    for (int i = 0; i < used; ++i) {
      const int s = kb - 1 - i;
      bar_wait(&bars.k_full[s < 0 ? s + KB : s], s < 0 ? kp : kp ^ 1u, err, ok ? kSpinCycles : kSpinCyclesAfterError);
    }
  } else if (warp >= C::kSumWarps) {
    // ---- what the keys of whole units have gathered, and their pages: a lane four keys (pages are 16 or more), the page
    // numbers of the next units under way
    struct Four {
      int key, head, page;
      bool held;  // some of them have gathered before
    };
    auto next_four = [&](Four& x) {
      do {
        if (!walk.next(a, g)) return false;
      } while (g.q.q_len == 0 || g.a != 0 || g.b != g.n);
      x.key = g.t * KT + 4 * lane;
      x.head = g.h;
      x.page = x.key < g.q.len ? __ldcg(a.table + int64_t(g.r) * a.width + (x.key >> a.page_shift)) : -1;
      x.held = x.key < g.q.held;
      return true;
    };
    int mb = 0;
    uint32_t mp = 1;
    KtAhead<Four, C::kAhead + 1> ahead;
    ahead.start(next_four);
    Four now;
    while (ok && ahead.take(now, next_four)) {
      ok = __all_sync(0xffffffffu, bar_wait(&bars.mark_empty[mb], mp, err));
      if (!ok) break;
      const bool there = now.page >= 0 && now.page < a.n_pages;
      s_page[mb * 32 + lane] = there ? now.page : -1;
      if (there && now.held)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sa(s_old + mb * 128 + 4 * lane)),
                     "l"(a.weight + ((int64_t(now.page) * a.hkv + now.head) << a.page_shift) + (now.key & ((1 << a.page_shift) - 1)))
                     : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sa(&bars.mark_full[mb])) : "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.mark_full[mb]);
      if (++mb == C::kMarks) mb = 0, mp ^= 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---- sums: a thread a key, the two warpgroups take the steps in turn
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const float scale = a.scale;
    const unsigned long long c2 = f2_pack(scale, scale), e2 = f2_pack(1.4426950408889634f, 1.4426950408889634f);
    int step = 0, pair = 0, marked = 0;  // steps, units of several steps, units with loaded marks so far
    auto wg_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
    while (walk.next(a, g)) {  // after a wait that gave up too: the warps meet at barriers
      const int key = g.t * KT + row;
      const int n_steps = g.q.q_len > 0 ? g.b - g.a : 0;
      const bool ends = wg == (n_steps > 0 ? (step + n_steps - 1) & 1 : 0);  // this warpgroup ends the part
      const bool whole = g.a == 0 && g.b == g.n, loaded = C::kFew && whole && n_steps > 0;
      const int mb = marked & 7;
      const uint32_t mp = uint32_t(marked >> 3) & 1u;
      marked += loaded;
      KwMark mark{-1, 0.f, 0};  // ahead of the wait for the scores
      if (loaded) {
        if (ends && a.offsets && (g.t + 1) * KT > g.q.held) mark.shift = __ldcg(a.offsets + g.r);
      } else if (ends) {
        mark = kw_mark(a, g, key);
      }
      unsigned long long acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
      for (int i = 0; i < n_steps; ++i, ++step) {
        if ((step & 1) != wg) continue;
        const int sb = step % SB;
        const uint32_t ph = uint32_t(step / SB) & 1u;
        const uint32_t s_at = tmem + lanes + sb * NR;
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
        // four rows' exponents from x on
        auto weights = [&](const uint32_t* sr, int x, float2& u, float2& v, int c) {
          const float4 l = *reinterpret_cast<const float4*>(lse + c + x);
          u = f2_unpack(f2_mul(f2_fma(f2_pack(__uint_as_float(sr[x]), __uint_as_float(sr[x + 1])), c2, f2_pack(l.x, l.y)), e2));
          v = f2_unpack(f2_mul(f2_fma(f2_pack(__uint_as_float(sr[x + 2]), __uint_as_float(sr[x + 3])), c2, f2_pack(l.z, l.w)), e2));
        };
        if (NR == 128 && !masked && n_rows == 128) {  // whole: a piece's scores are loaded while the one before is added
          uint32_t sr[2][32];
          tl_ld32(s_at, sr[0]);
          tl_wait_ld();
          tl_arrived32(sr[0]);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            if (p < 3) tl_ld32(s_at + 32 * (p + 1), sr[(p + 1) & 1]);
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              float2 u, v;
              weights(sr[p & 1], x, u, v, 32 * p);
              acc[0] = f2_add(acc[0], f2_pack(ex2(u.x), ex2(u.y)));
              acc[1] = f2_add(acc[1], f2_pack(ex2(v.x), ex2(v.y)));
            }
            if (p < 3) {
              tl_wait_ld();
              tl_arrived32(sr[(p + 1) & 1]);
            }
          }
        } else
#pragma unroll 1
        for (int c = 0; c < n_rows; c += CH) {
          uint32_t sr[CH];
          if constexpr (CH == 16) {
            kt_ld16(s_at + c, sr);
            tl_wait_ld();
            kt_arrived16(sr);
          } else {
            tl_ld32(s_at + c, sr);
            tl_wait_ld();
            tl_arrived32(sr);
          }
          if (!masked && c + CH <= n_rows) {
#pragma unroll
            for (int x = 0; x < CH; x += 4) {
              float2 u, v;
              weights(sr, x, u, v, c);
              acc[0] = f2_add(acc[0], f2_pack(ex2(u.x), ex2(u.y)));
              acc[1] = f2_add(acc[1], f2_pack(ex2(v.x), ex2(v.y)));
            }
          } else {  // a bit a row: those from `from` on that lie before `to`
            const int from = late - c, to = n_rows - c;
            const uint32_t below_to = to >= 32 ? ~0u : (1u << to) - 1u;
            const uint32_t see = from >= 32 ? 0u : from <= 0 ? below_to : below_to & ~((1u << from) - 1u);
#pragma unroll
            for (int x = 0; x < CH; x += 4) {
              float2 u, v;
              weights(sr, x, u, v, c);
              if (!(see >> x & 1u)) u.x = -INFINITY;
              if (!(see >> (x + 1) & 1u)) u.y = -INFINITY;
              if (!(see >> (x + 2) & 1u)) v.x = -INFINITY;
              if (!(see >> (x + 3) & 1u)) v.y = -INFINITY;
              acc[0] = f2_add(acc[0], f2_pack(ex2(u.x), ex2(u.y)));
              acc[1] = f2_add(acc[1], f2_pack(ex2(v.x), ex2(v.y)));
            }
          }
        }
        tl_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.s_empty[sb]);
      }
      const float2 s01 = f2_unpack(f2_add(acc[0], acc[1]));
      float sum = s01.x + s01.y;
      if (n_steps > 1) {  // the other warpgroup's steps
        float* theirs = s_half + (pair & 1) * 128;
        ++pair;
        if (!ends) theirs[row] = sum;
        asm volatile("bar.sync 3, 256;" ::: "memory");
        if (ends) sum += theirs[row];
      }
      if (loaded) {
        // Both warpgroups wait for the marks and give their place in the ring back: the next unit there may be the other one's,
        // and a parity tells a phase from its neighbours only.
        ok = ok && __all_sync(0xffffffffu, bar_wait(&bars.mark_full[mb], mp, err));
        if (!ok) continue;
        mark.old = s_old[mb * 128 + row];
        const int pg = s_page[mb * 32 + row / 4];
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.mark_empty[mb]);
        if (pg >= 0 && key < g.q.len) mark.at = ((int64_t(pg) * a.hkv + g.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
      }
      if (!ends) continue;
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
        kw_give(a, g, key, mark, sum);
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
  if (e == cudaSuccess) e = attn_page_map(&mk, m, a.K, page < 128 ? page : 128);
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
