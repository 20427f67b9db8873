// Attention of many query rows (prompts, chunks, grouped heads): row tiles of
// 128 on the tensor cores (tcgen05, TMEM), sm_103a.

#include "gsi_attn.cuh"

namespace gsi {

// A unit is NQ row tiles of 128 query rows (floor(128 / G) tokens of the G
// heads that share a key/value head), over tiles of 128 keys:
//   S = Q K^T (tcgen05, both operands in shared memory, S in TMEM)
//   p = 2^(S c - m), l += sum p, per row; where m grows by more than 2^8 the
//       output so far is scaled to the new m (below that the larger weights
//       stay within bf16 and float32 range and the scaling is saved)
//   O += P V (P bf16 in TMEM over the columns of S, V in shared memory)
// Roles: one thread issues every product; a copy warp fills a ring of 32 KB
// stages by TMA (a K stage is 128 columns of the tile's 128 keys, a V stage all
// columns of 64 or 128 keys), in the order in which the products use them; a
// warpgroup a row tile owns the softmax (a thread a row, so neither maximum
// nor sum needs an exchange); two warps clean the masked tiles' V (below).
// Up to 128 columns NQ = 2: the products of one row tile run while the other
// one's softmax does, and each key is read from L2 once for 256 rows.  Above,
// the output of one tile takes half of TMEM, and two S buffers of one row tile
// alternate instead.
//
// What bounds it: up to 128 columns the chain of a row tile (S, its maximum, 128
// exponentials a thread, then its two products, ~3000 cycles a tile of 256 rows
// against 2048 of products); above, the reads of L2 (128 KB a tile of 128 rows,
// ~10 TB/s over the SMs).  8192 tokens: 32 x 128 403 us (1.36 PFLOP/s), 16 x 256
// 422 us (1.30), 32 x 64 364 us (0.76); 2048 tokens of 16 x 256 42 us.
//
// Masked tiles: S is masked in registers; a weight of 0 hides a number of V
// but not an infinity or NaN, nor the ring's stale bytes where no page was
// copied, so those values are set to zero in shared memory before the product
// and the non-finite ones that a row does see are added at its end.
constexpr int kTileKeys = 128;
constexpr int kSlabBytes = 16384;  // 64 columns of 128 rows
// What a unit costs beside its tiles, in tiles (its queries' load and its rows' output), and a part of one to write and fold.
constexpr int kTileUnit = 2;

template <int NS>
struct TilesCfg {
  static constexpr int kNQ = NS <= 2 ? 2 : 1;
  static constexpr int kStage = NS == 1 ? kSlabBytes : 2 * kSlabBytes;
  static constexpr int kKST = (NS + 1) / 2;             // stages of a K tile: two slabs each
  static constexpr int kVST = kKST;                     // stages of a V tile
  static constexpr int kVK = kTileKeys / kVST;          // keys of a V stage
  static constexpr int kSoftWarps = 4 * kNQ;
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  static constexpr int kQBytes = kNQ * NS * kSlabBytes;
  static constexpr int kStages = (232448 - 2048 - kQBytes) / kStage;
  static constexpr size_t kSmem = 1024 + size_t(kQBytes) + size_t(kStages) * kStage + 1024;
  static constexpr int kOCol = 256;  // TMEM: S buffers at 0 and 128, O from here
  static_assert(NS * 128 * kVK <= kStage, "V stages");
  static_assert(kStages >= 2 * kKST + 1, "a K and a V tile, and one stage ahead");
  static_assert(kOCol + kNQ * NS * 64 <= 512, "TMEM columns");
};

struct TilesBars {
  uint64_t full[12], empty[12];
  uint64_t dirty, clean;  // a masked tile's V is there; it is cleaned
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], o_free[2];
  uint64_t q_full, done;
  uint32_t tmem;
  int found[8];  // per segment (mod 8): its number + 1 where a non-finite value was taken out
  int last[2];
};
static_assert(sizeof(TilesBars) <= 1024, "barriers");

// Place in the ring: stage and phase parity.
template <int N>
struct TilesRing {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step(int n) {
    s += n;
    if (s >= N) {
      s -= N;
      ph ^= 1;
    }
  }
  __device__ __forceinline__ TilesRing at(int n) const {
    TilesRing r = *this;
    r.step(n);
    return r;
  }
};

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void tl_mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}
__device__ __forceinline__ void tl_mma_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(at), "l"(bd), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}
// One lane of the warp.  (The compiler knows that a branch on this has one
// thread, and the products' operands then reach their uniform registers
// directly; behind `lane == 0` it loops over the threads there might be, at
// ~190 cycles a product.)
__device__ __forceinline__ bool tl_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tl_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sa(bar)) : "memory");
}
__device__ __forceinline__ void tl_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tl_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tl_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tl_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define GSI_R8(r, i) "=r"((r)[(i)]), "=r"((r)[(i) + 1]), "=r"((r)[(i) + 2]), "=r"((r)[(i) + 3]), "=r"((r)[(i) + 4]), \
                     "=r"((r)[(i) + 5]), "=r"((r)[(i) + 6]), "=r"((r)[(i) + 7])
#define GSI_W8(r, i) "r"((r)[(i)]), "r"((r)[(i) + 1]), "r"((r)[(i) + 2]), "r"((r)[(i) + 3]), "r"((r)[(i) + 4]), \
                     "r"((r)[(i) + 5]), "r"((r)[(i) + 6]), "r"((r)[(i) + 7])
// 32 columns of this warp's 32 lanes (no wait).
__device__ __forceinline__ void tl_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%32];"
      : GSI_R8(r, 0), GSI_R8(r, 8), GSI_R8(r, 16), GSI_R8(r, 24)
      : "r"(t));
}
__device__ __forceinline__ void tl_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(t), GSI_W8(r, 0), GSI_W8(r, 8), GSI_W8(r, 16), GSI_W8(r, 24)
      : "memory");
}

// After tl_wait_ld(): nothing that uses these registers may move before it.
#define GSI_H8(r, i) "+r"((r)[(i)]), "+r"((r)[(i) + 1]), "+r"((r)[(i) + 2]), "+r"((r)[(i) + 3]), "+r"((r)[(i) + 4]), \
                     "+r"((r)[(i) + 5]), "+r"((r)[(i) + 6]), "+r"((r)[(i) + 7])
__device__ __forceinline__ void tl_arrived32(uint32_t* r) {
  asm volatile("" : GSI_H8(r, 0), GSI_H8(r, 8), GSI_H8(r, 16), GSI_H8(r, 24)::"memory");
}

// Shared-memory operand descriptors, 128-byte swizzle (version 1).  K-major
// (Q, K: rows of 64 columns): 8-row groups 1024 bytes apart.  MN-major (V: a
// row is a key, its 64 columns run along N): 8-key groups 1024 bytes apart,
// the next 64 columns `slab` bytes on.
__device__ __forceinline__ uint64_t tl_desc(uint32_t addr, uint32_t slab) {
  return uint64_t((addr & 0x3ffffu) >> 4) | (uint64_t(slab >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// kind::f16, A and B bf16, D float32; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t tl_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

__device__ __forceinline__ void tl_load_query(uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, int head, int tok) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(col), "r"(head), "r"(tok), "r"(bar)
      : "memory");
}

// What every role derives from a segment: the row tiles' tokens and key ranges.
template <int NQ>
struct TilesSeg {
  int tok0[NQ], n_tok[NQ];  // tokens of each row tile
  int ja[NQ], jb[NQ];       // the segment's tiles (of the unit) that some row of it sees
  int lo_all, lim_all;      // keys that some row of the unit sees
  int lo_max, lim_min;      // keys that every row of the unit sees lie in [lo_max, lim_min)
  __device__ __forceinline__ void set(const AttnArgs& a, const AttnSeg& g, int tpt) {
    const int u0 = g.u * NQ * tpt, u1 = min(u0 + NQ * tpt, g.q.q_len);
    lim_min = attn_lim(a, g.q, u0);
    lim_all = attn_lim(a, g.q, u1 - 1);
    lo_all = attn_lo(a, lim_min);
    lo_max = attn_lo(a, lim_all);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      tok0[q] = u0 + q * tpt;
      n_tok[q] = max(0, min(tpt, u1 - tok0[q]));
      ja[q] = jb[q] = g.a;
      if (n_tok[q] > 0 && g.b > g.a) {
        const int lim = attn_lim(a, g.q, tok0[q] + n_tok[q] - 1), lo = attn_lo(a, attn_lim(a, g.q, tok0[q]));
        ja[q] = max(g.a, lo / kTileKeys - g.t0);
        jb[q] = min(g.b, (lim + kTileKeys - 1) / kTileKeys - g.t0);
        if (jb[q] <= ja[q]) ja[q] = jb[q] = g.a;
      }
    }
  }
  __device__ __forceinline__ bool sees(int q, int j) const { return j >= ja[q] && j < jb[q]; }
  // some row does not see some key of tile t
  __device__ __forceinline__ bool masked(int t) const { return t * kTileKeys < lo_max || (t + 1) * kTileKeys > lim_min; }
};

template <int NS>
__global__ void __launch_bounds__(TilesCfg<NS>::kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnArgs a) {
  using C = TilesCfg<NS>;
  constexpr int NQ = C::kNQ, VK = C::kVK, KST = C::kKST, VST = C::kVST, STAGES = C::kStages;
  using Ring = TilesRing<STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = base;
  uint8_t* ring = base + C::kQBytes;
  TilesBars& bars = *reinterpret_cast<TilesBars*>(ring + STAGES * C::kStage);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      bar_init(&bars.full[s], 1);
      bar_init(&bars.empty[s], 1);
    }
    bar_init(&bars.dirty, 1);
    bar_init(&bars.clean, 2);
    for (int q = 0; q < 2; ++q) {
      bar_init(&bars.s_full[q], 1);
      bar_init(&bars.p_half[q], 4);
      bar_init(&bars.p_full[q], 4);
      bar_init(&bars.pv_done[q], 1);
      bar_init(&bars.o_free[q], 4);
    }
    bar_init(&bars.q_full, 1);
    bar_init(&bars.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mq) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mk) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mv) : "memory");
    for (int i = 0; i < 8; ++i) bars.found[i] = 0;
  }
  if (warp == C::kSoftWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&bars.tmem)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tl_fence_before();
  pdl_wait();
  const int tpt = 128 / a.group, ut = NQ * tpt;
  AttnWalk walk;
  walk.ut = ut;
  walk.kt = kTileKeys;
  walk.s = attn_share<C::kThreads>(a, ut, kTileKeys, kTileUnit, walk.p);  // its block barriers publish the ones above
  tl_fence_after();
  const uint32_t tmem = bars.tmem;
  uint32_t* err = attn_err(a);
  AttnSeg g;
  TilesSeg<NQ> t;
  bool ok = true;

  if (warp >= C::kSoftWarps) {
    if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == C::kSoftWarps) {
      // ---- the products (one thread)
      if (tl_elect()) {
        constexpr uint32_t id_qk = tl_idesc(kTileKeys, false), id_pv = tl_idesc(NS * 64, true);
        const uint64_t dq = tl_desc(sa(s_q), 0), dk = tl_desc(sa(ring), 0), dv = tl_desc(sa(ring), VK * 128);
        constexpr uint64_t kStageD = C::kStage / 16, kSlabD = kSlabBytes / 16;
        Ring r;
        uint32_t ph_q = 0, ph_clean = 0, ph_p[2] = {0, 0}, ph_o[2] = {1, 1};  // the first wait for a free O passes
        uint32_t buf1 = 0;  // one row tile: the S buffer of the tile
        auto load_q = [&]() {
          t.set(a, g, tpt);
          if (g.b == g.a) return;
          const int tiles = NQ == 2 && t.n_tok[NQ - 1] > 0 ? 2 : 1;
          bar_expect_tx(&bars.q_full, uint32_t(tiles * NS * tpt * a.group) * 128);
          for (int q = 0; q < tiles; ++q)
            for (int s = 0; s < NS; ++s)
              tl_load_query(sa(s_q + (q * NS + s) * kSlabBytes), &mq, sa(&bars.q_full), s * 64, g.h * a.group,
                            g.q.q0 + t.tok0[0] + q * tpt);
        };
        auto wait_full = [&](const Ring& x) {
          ok = ok && bar_wait(&bars.full[x.s], x.ph, err);
          tl_fence_after();
        };
        // the V stages at x are there, and cleaned
        auto wait_v = [&](const Ring& x, bool masked) {
#pragma unroll
          for (int i = 0; i < VST; ++i) wait_full(x.at(i));
          if (masked && ok) {
            bar_arrive(&bars.dirty);
            ok = bar_wait(&bars.clean, ph_clean, err);
            ph_clean ^= 1;
            tl_fence_after();
          }
        };
        auto release = [&](const Ring& x, int n) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (i < n) tl_commit(&bars.empty[x.at(i).s]);
        };
        // S[buf] = Q_q K^T, K in the stages at x
        auto qk = [&](int q, uint32_t buf, const Ring& x) {
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const uint64_t ad = dq + uint64_t(q * NS + s) * kSlabD;
            const uint64_t bd = dk + uint64_t(x.at(s / 2).s) * kStageD + uint64_t(s % 2) * kSlabD;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tl_mma_ss(tmem + buf * 128, ad + uint64_t(2 * k), bd + uint64_t(2 * k), id_qk, (s | k) != 0);
          }
          tl_commit(&bars.s_full[buf]);
        };
        // O_q += P[buf] V, V in the stages at x.  (Issued by one thread, the products run in order: S[buf] may be
        // written again by the next one.)
        // The weights of the first 64 keys come first, so half of the product runs while the others are formed.
        auto pv = [&](int q, uint32_t buf, uint32_t parity, const Ring& x, bool first) {
          ok = ok && bar_wait(&bars.p_half[buf], parity, err);
          tl_fence_after();
          if (!ok) return;
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k) {
            if (k == kTileKeys / 32) {
              ok = bar_wait(&bars.p_full[buf], parity, err);
              tl_fence_after();
              if (!ok) return;
            }
            const uint64_t bd = dv + uint64_t(x.at(k * 16 / VK).s) * kStageD + uint64_t((k * 16 % VK) * 8);
            tl_mma_ts(tmem + C::kOCol + q * 128, tmem + buf * 128 + k * 8, bd, id_pv, !(first && k == 0));
          }
        };
        auto wait_o = [&](int q) {
          ok = ok && bar_wait(&bars.o_free[q], ph_o[q], err);
          ph_o[q] ^= 1;
        };
        bool have = walk.next(a, g);
        if (have) load_q();
        while (ok && have) {
          if (g.b > g.a) {
            ok = bar_wait(&bars.q_full, ph_q, err);
            ph_q ^= 1;
            tl_fence_after();
#pragma unroll
            for (int i = 0; i < KST; ++i) wait_full(r.at(i));
            if constexpr (NQ == 2) {
              if (ok) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  if (t.sees(q, g.a)) qk(q, q, r);
                release(r, 1);
              }
              r.step(1);
              for (int j = g.a; ok && j < g.b; ++j) {
                const Ring v = r, k = r.at(1);
                const bool more = j + 1 < g.b;
                wait_v(v, t.masked(g.t0 + j));
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  if (t.sees(q, j)) {
                    const bool first = j == t.ja[q];
                    if (first) wait_o(q);
                    if (ok) pv(q, q, ph_p[q], v, first);
                    ph_p[q] ^= 1;
                    if (ok && j + 1 == t.jb[q]) tl_commit(&bars.pv_done[q]);
                  }
                  if (q == 1 && ok) release(v, 1);
                  if (q == 0 && more) wait_full(k);
                  if (more && ok && t.sees(q, j + 1)) qk(q, q, k);
                }
                if (more && ok) release(k, 1);
                r.step(more ? 2 : 1);
              }
            } else {
              if (ok) {
                qk(0, buf1, r);
                release(r, KST);
              }
              r.step(KST);
              for (int j = g.a; ok && j < g.b; ++j) {
                if (j + 1 < g.b) {
#pragma unroll
                  for (int i = 0; i < KST; ++i) wait_full(r.at(i));
                  if (!ok) break;
                  qk(0, buf1 ^ 1, r);
                  release(r, KST);
                  r.step(KST);
                }
                wait_v(r, t.masked(g.t0 + j));
                const bool first = j == g.a;
                if (first) wait_o(0);
                if (ok) pv(0, buf1, buf1 ? ph_p[1] : ph_p[0], r, first);
                if (!ok) break;
                if (buf1) ph_p[1] ^= 1; else ph_p[0] ^= 1;
                tl_commit(&bars.pv_done[0]);
                release(r, VST);
                r.step(VST);
                buf1 ^= 1;
              }
            }
          }
          // every S of this segment has been read, so Q may be replaced
          have = walk.next(a, g);
          if (ok && have) load_q();
        }
        tl_commit(&bars.done);
        bar_wait(&bars.done, 0, err, ok ? kSpinCycles : kSpinCyclesAfterError);
        if (!ok) bar_wait(&bars.q_full, ph_q, err, kSpinCyclesAfterError);
      }
      __syncwarp();
    } else if (warp == C::kSoftWarps + 1) {
      // ---- copies: lane l issues box l of a stage (at most 16)
      const int page = 1 << a.page_shift;
      const int bk = min(page, kTileKeys), bv = min(page, VK);
      Ring r;
      uint32_t used = 0;  // stages filled so far, up to STAGES
      // the copy of one stage: K columns from slab 2 `part`, or V keys from VK `part`; pid: lane i has the tile's page i
      auto copy = [&](bool is_v, int part, int key0, int pid) {
        const int rows = is_v ? bv : bk, per = (is_v ? VK : kTileKeys) / rows;  // boxes of 64 columns
        const int b = lane % per, slab = lane / per;
        const int row0 = (is_v ? part * VK : 0) + b * rows;  // in the tile
        const int col = is_v ? slab : 2 * part + slab;       // slab of the row
        const bool mine = slab < (is_v ? NS : 2) && col < NS && key0 + row0 < t.lim_all && key0 + row0 + rows > t.lo_all;
        const int id = __shfl_sync(0xffffffffu, pid, page >= kTileKeys ? 0 : row0 >> a.page_shift);
        if (used == STAGES) ok = __all_sync(0xffffffffu, bar_wait(&bars.empty[r.s], r.ph ^ 1u, err)); else ++used;
        if (!ok) return;
        const uint32_t bytes = uint32_t(rows) * 128;
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) bar_expect_tx(&bars.full[r.s], uint32_t(n) * bytes);
        __syncwarp();
        if (mine)
          tma_load_page(sa(ring + r.s * C::kStage) + slab * (is_v ? VK * 128 : kSlabBytes) + b * bytes, is_v ? &mv : &mk,
                        sa(&bars.full[r.s]), col * 64, (key0 + row0) & (page - 1), g.h, id);
        r.step(1);
      };
      while (ok && walk.next(a, g)) {
        t.set(a, g, tpt);
        const int32_t* row = a.table + int64_t(g.r) * a.width;
        auto page_of = [&](int j) {  // lane i: page i of tile j (0 where no row sees it)
          const int k = (g.t0 + j) * kTileKeys + lane * page;
          return j < g.b && lane * page < kTileKeys && k < t.lim_all && k + page > t.lo_all ? __ldcg(row + (k >> a.page_shift)) : 0;
        };
        int pid = page_of(g.a);
        if (NQ == 1 && g.b > g.a)
          for (int i = 0; ok && i < KST; ++i) copy(false, i, (g.t0 + g.a) * kTileKeys, pid);
        for (int j = g.a; ok && j < g.b; ++j) {
          const int next = page_of(j + 1);
          const int key0 = (g.t0 + j) * kTileKeys;
          if (NQ == 2)
            copy(false, 0, key0, pid);
          else if (j + 1 < g.b)
            for (int i = 0; ok && i < KST; ++i) copy(false, i, key0 + kTileKeys, next);
          for (int i = 0; ok && i < VST; ++i) copy(true, i, key0, pid);
          pid = next;
        }
      }
      // the copies in flight land before the CTA leaves: the last use of every stage that was filled
      for (uint32_t i = 0; i < used; ++i) {
        // going back from r: stage r.s - 1 - i, in the phase before r's once the ring has wrapped
        const int s = r.s - 1 - int(i);
        bar_wait(&bars.full[s < 0 ? s + STAGES : s], s < 0 ? r.ph ^ 1u : r.ph, err, ok ? kSpinCycles : kSpinCyclesAfterError);
      }
    } else {
      // ---- masked tiles' V: what lies outside the unit's keys, or is not finite, becomes zero
      const int ct = tid - 32 * (C::kSoftWarps + 2);  // 0 .. 63
      int p = 0, seg = 0;  // stages before this segment
      uint32_t ph = 0;
      while (ok && walk.next(a, g)) {
        t.set(a, g, tpt);
        for (int j = g.a; ok && j < g.b; ++j) {
          if (!t.masked(g.t0 + j)) continue;
          // the V stages of tile j, in the order of the copies
          const int vs = p + KST + (j - g.a) * (KST + VST) + (NQ == 1 && j + 1 < g.b ? KST : 0);
          const int key0 = (g.t0 + j) * kTileKeys;
          bool found = false;
          ok = __all_sync(0xffffffffu, bar_wait(&bars.dirty, ph, err));
          ph ^= 1;
          if (!ok) break;
          for (int v = 0; v < VST; ++v) {
            uint8_t* sl = ring + (vs + v) % STAGES * C::kStage;
            // 16-byte pieces, eight in flight a thread; a row (key) is 128 bytes of a slab
            const bool inside = key0 >= t.lo_all && key0 + kTileKeys <= t.lim_all;
#pragma unroll 1
            for (int e0 = ct; e0 < NS * VK * 8; e0 += 64 * 8) {
              uint4 y[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) y[x] = reinterpret_cast<const uint4*>(sl)[e0 + 64 * x];
              uint32_t bad = 0;  // an exponent of all ones carries into the sign bit
#pragma unroll
              for (int x = 0; x < 8; ++x)
                bad |= ((y[x].x & 0x7f807f80u) + 0x00800080u) | ((y[x].y & 0x7f807f80u) + 0x00800080u) |
                       ((y[x].z & 0x7f807f80u) + 0x00800080u) | ((y[x].w & 0x7f807f80u) + 0x00800080u);
              const bool some_bad = (bad & 0x80008000u) != 0;
              if (inside && !some_bad) continue;
#pragma unroll 1
              for (int e = e0; e < e0 + 64 * 8; e += 64) {
                const int key = key0 + v * VK + (e >> 3) % VK;
                if (key < t.lo_all || key >= t.lim_all) {
                  reinterpret_cast<uint4*>(sl)[e] = make_uint4(0, 0, 0, 0);
                } else if (some_bad) {
                  uint32_t* w = reinterpret_cast<uint32_t*>(sl) + 4 * e;
#pragma unroll 1
                  for (int z = 0; z < 4; ++z) {
                    const uint32_t keep = ((w[z] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) |
                                          ((w[z] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
                    if (keep != 0xffffffffu) {
                      w[z] &= keep;
                      found = true;
                    }
                  }
                }
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // these writes, before the product reads
          if (found) bars.found[seg & 7] = seg + 1;
          __syncwarp();
          if (lane == 0) bar_arrive(&bars.clean);
        }
        p += (g.b - g.a) * (KST + VST);
        ++seg;
      }
    }
  } else {
    // ---- softmax: a warpgroup a row tile, a thread a row
    if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int q = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);  // powers of two; a scale of 0 still masks
    const bool neg = a.scale < 0.f;
    const uint32_t o_at = tmem + lanes + C::kOCol + q * 128;
    int ks = 0, seg = 0;
    uint32_t ph_pv = 0;  // two row tiles: the segments that ended
    // One row tile: the product of the tile before number ks is done.  A parity tells one phase from its neighbours only,
    // so every phase is seen: a tile's weights are handed over whole (its own product cannot end before) after the
    // product of the tile before, and at the segment's end just the last one is out.
    auto product_before = [&]() {
      return ks == 0 || __all_sync(0xffffffffu, bar_wait(&bars.pv_done[0], uint32_t(ks - 1) & 1u, err));
    };
    while (walk.next(a, g)) {  // after a wait that gave up too: the warps of a row tile meet at barriers
      t.set(a, g, tpt);
      const int this_seg = seg++;
      const int tok0 = q == 0 ? t.tok0[0] : t.tok0[NQ - 1], n_tok = q == 0 ? t.n_tok[0] : t.n_tok[NQ - 1];
      const int ja = q == 0 ? t.ja[0] : t.ja[NQ - 1], jb = q == 0 ? t.jb[0] : t.jb[NQ - 1];
      if (n_tok == 0) continue;
      const int n_rows = n_tok * a.group;
      const int my_tok = tok0 + min(row / a.group, n_tok - 1);
      const int lim = attn_lim(a, g.q, my_tok), lo = attn_lo(a, lim);
      const int lim_min = attn_lim(a, g.q, tok0), lo_max = attn_lo(a, attn_lim(a, g.q, tok0 + n_tok - 1));
      float m = -INFINITY, l = 0.f;  // m in units of S; weights are 2^(c (S - m))
      for (int j = ja; j < jb; ++j, ++ks) {
        const int buf = NQ == 2 ? q : ks & 1;
        const uint32_t s_at = tmem + lanes + buf * 128;
        ok = ok && __all_sync(0xffffffffu, bar_wait(&bars.s_full[buf], uint32_t(NQ == 2 ? ks : ks >> 1) & 1u, err));
        if (!ok) continue;
        tl_fence_after();
        uint32_t sr[128];
        float* s = reinterpret_cast<float*>(sr);
#pragma unroll
        for (int i = 0; i < 4; ++i) tl_ld32(s_at + 32 * i, sr + 32 * i);
        tl_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) tl_arrived32(sr + 32 * i);
        const int tile = (g.t0 + j) * kTileKeys;
        if (neg) {
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] = -s[i];
        }
        if (tile < lo_max || tile + kTileKeys > lim_min) {
          // a bit a key: those from `from` on that lie before `to`
          const int from = lo - tile, to = lim - tile;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t below_to = to >= 32 * w + 32 ? ~0u : to <= 32 * w ? 0u : (1u << (to - 32 * w)) - 1u;
            const uint32_t below_from = from >= 32 * w + 32 ? ~0u : from <= 32 * w ? 0u : (1u << (from - 32 * w)) - 1u;
            const uint32_t see = below_to & ~below_from;
#pragma unroll
            for (int i = 0; i < 32; ++i) s[32 * w + i] = (see >> i) & 1u ? s[32 * w + i] : -INFINITY;
          }
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int z = 0; z < 4; ++z) mx[z] = max3(mx[z], s[i + 2 * z], s[i + 2 * z + 1]);
        const float m_new = max3(max3(mx[0], mx[1], m), max3(mx[2], mx[3], s[124]), max3(s[125], s[126], s[127]));
        // (m_new - m is NaN where both are infinite: nothing to scale)
        if (__any_sync(0xffffffffu, (m_new - m) * c > 8.f)) {
          const float f = m == -INFINITY ? 0.f : ex2((m - m_new) * c);
          m = m_new;
          l *= f;
          if (j > ja) {
            // O has to be complete up to the tile before.  With two row tiles this S was made after that product.
            if constexpr (NQ == 1) {
              ok = product_before();
              if (!ok) continue;
              tl_fence_after();
            }
#pragma unroll 1
            for (int i = 0; i < NS * 2; ++i) {
              uint32_t r[32];
              tl_ld32(o_at + 32 * i, r);
              tl_wait_ld();
              tl_arrived32(r);
#pragma unroll
              for (int z = 0; z < 32; ++z) r[z] = __float_as_uint(__uint_as_float(r[z]) * f);
              tl_st32(o_at + 32 * i, r);
            }
          }
        }
        float mc = m == -INFINITY ? 0.f : m * c;
        // S c - m c as one fused product is off by up to |m c| 2^-24, at large scores more than S itself is where the
        // scores are alike: subtract first there
        if (__any_sync(0xffffffffu, fabsf(mc) > 256.f)) {
          const float d = mc == 0.f ? 0.f : m;
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] -= d;
          mc = 0.f;
        }
        const unsigned long long c2 = f2_pack(c, c), mc2 = f2_pack(-mc, -mc);
        // weights of the keys from i0 on; they enter the second product as bf16 (2^-8 of each at most, like the
        // cache's own rounding), and what enters it is what is summed: the output is a mean of the values for any
        // rounding
        auto weights = [&](int i0, int n, uint32_t* pr) {
#pragma unroll
          for (int i = 0; i < n; i += 2) {
            float2 w = f2_unpack(f2_fma(f2_pack(s[i0 + i], s[i0 + i + 1]), c2, mc2));
            w.x = ex2(w.x);
            w.y = ex2(w.y);
            pr[i / 2] = attn_pack(w.x, w.y);
          }
        };
        auto give = [&](uint64_t* bar) {
          tl_wait_st();
          tl_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(bar);
        };
        uint32_t pr[32];
        weights(0, 64, pr);
        tl_st32(s_at, pr);
        uint32_t pr2[32];
        weights(64, 32, pr2);
        give(&bars.p_half[buf]);
        weights(96, 32, pr2 + 16);
        tl_st32(s_at + 32, pr2);
        if constexpr (NQ == 1) {
          ok = product_before();
          if (!ok) continue;
        }
        give(&bars.p_full[buf]);
        // The weights that entered the product are summed behind their hand-over: the chain up to it is what bounds a tile.
        // Against a sum of the weights before their rounding this costs, us: 5 chunks of 509 tokens over 8003 keys 146
        // (144), 8192 tokens of 32 x 128 402 (399), of 16 x 256 427 (420), of 32 x 64 361 (346); with the sum ahead of the
        // hand-over 150, 415, 430, 370.
        float sum[4] = {};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          add_bf16x2(sum[0], sum[1], pr[i]);
          add_bf16x2(sum[2], sum[3], pr2[i]);
        }
        l += (sum[0] + sum[2]) + (sum[1] + sum[3]);
      }

      // ---- the segment's end: the rows are finished, or left as a part
      const bool some = jb > ja;
      if (some && ok) {
        if constexpr (NQ == 2) {
          ok = __all_sync(0xffffffffu, bar_wait(&bars.pv_done[q], ph_pv, err));
          ph_pv ^= 1;
        } else {
          ok = product_before();
        }
        tl_fence_after();
      }
      const bool whole = g.a == 0 && g.b == g.n;
      const bool any = some && *reinterpret_cast<volatile int*>(&bars.found[this_seg & 7]) == this_seg + 1;
      int b0, b1;
      walk.parts(g, b0, b1);
      const float ml = m == -INFINITY ? m : m * c;  // the parts' maxima are in powers of two
      const unsigned n_parts = unsigned(b1 - b0 + 1);
      auto wg_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory"); };
      // The part that begins a unit is the last thing its CTA does and the others' first, so they are there as a
      // rule: then they are folded in here, and nothing of this one is written.  (A thread folds its row's parts one
      // after the other; many parts are joined faster by all threads.)
      bool fold = false;
      if (!whole && b0 == int(blockIdx.x) && n_parts <= 4) {
        if ((warp & 3) == 0 && lane == 0) {
          unsigned n;
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(attn_counter(a, b0, q)) : "memory");
          bars.last[q] = n == n_parts - 1;
          if (n == n_parts - 1) *attn_counter(a, b0, q) = 0;
        }
        wg_sync();
        fold = *reinterpret_cast<volatile int*>(&bars.last[q]) != 0;
        wg_sync();
      }
      if (any && ok) {
#pragma unroll 1
        for (int i = 0; i < a.dim; ++i) {
          uint32_t x;
          __syncwarp();
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(o_at + i));
          tl_wait_ld();
          asm volatile("" : "+r"(x)::"memory");
          if (row < n_rows)
            x = __float_as_uint(attn_nonfinite<BF16>(a, g, kTileKeys, lo, lim, t.lo_max, t.lim_min, i, __uint_as_float(x)));
          __syncwarp();
          asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(o_at + i), "r"(x) : "memory");
          tl_wait_st();
        }
      }
      float* part = attn_part(a, 2 * int(blockIdx.x) + (int(blockIdx.x) == b0), NQ, q, 128);
      const int64_t out = row < n_rows ? attn_out_row(a, g, tok0, row) * a.dim : 0;
#pragma unroll 1
      for (int i = 0; i < NS; ++i) {
        uint32_t r[64];
        __syncwarp();
        if (some && ok) {
          tl_ld32(o_at + 64 * i, r);
          tl_ld32(o_at + 64 * i + 32, r + 32);
          tl_wait_ld();
          tl_arrived32(r);
          tl_arrived32(r + 32);
        } else {
#pragma unroll
          for (int z = 0; z < 64; ++z) r[z] = 0;
        }
        if (row < n_rows) {
          float v[64];
#pragma unroll
          for (int z = 0; z < 64; ++z) v[z] = __uint_as_float(r[z]);
          if (whole || fold) {
            float fm = ml, fl = l;
            if (fold) attn_fold<false, 64>(a, b0 + 1, b1, b0, NQ, q, 128, row, 64 * i, fm, fl, v);
            attn_finish<BF16, 64>(a, g.q, my_tok, out + 64 * i, 64 * i, fl, v);
          } else {
#pragma unroll
            for (int z = 0; z < 64; z += 4)
              if (64 * i + z < a.dim)
                *attn_piece<false>(part, 128, a.dim, row, 64 * i + z) = make_float4(v[z], v[z + 1], v[z + 2], v[z + 3]);
          }
        }
      }
      __syncwarp();
      if (some) {
        tl_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.o_free[q]);
      }
      if (!whole && !fold) {
        if (row < n_rows) {
          part[row] = ml;
          part[128 + row] = l;
        }
        __threadfence();
        wg_sync();
        if ((warp & 3) == 0 && lane == 0) {
          const bool last = atomicAdd(attn_counter(a, b0, q), 1u) == n_parts - 1;
          if (last) *attn_counter(a, b0, q) = 0;
          bars.last[q] = last;
        }
        wg_sync();
        const bool last = *reinterpret_cast<volatile int*>(&bars.last[q]) != 0;
        if (last) {
          __threadfence();
          // few rows: eight columns a thread, eight parts in flight
          if (n_rows <= 32)
            attn_join<BF16, false, 8>(a, g, b0, b1, NQ, q, 128, n_rows, tok0, row, 128);
          else
            attn_join<BF16, false, 64>(a, g, b0, b1, NQ, q, 128, n_rows, tok0, row, 128);
        }
        wg_sync();  // before the flag is written again
      }
    }
  }
  tl_fence_before();
  __syncthreads();
  if (warp == C::kSoftWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <int NS>
static cudaError_t launch_tiles(const AttnArgs& a, cudaStream_t s) {
  using C = TilesCfg<NS>;
  static_assert(C::kSmem <= 232448 && C::kStages <= 12, "shared memory of an SM");
  const int page = 1 << a.page_shift;
  CUtensorMap mq, mk, mv;
  cudaError_t e = attn_query_map(&mq, a, a.group, 128 / a.group);
  if (e == cudaSuccess) e = attn_page_map(&mk, a, a.K, page < kTileKeys ? page : kTileKeys);
  if (e == cudaSuccess) e = attn_page_map(&mv, a, a.V, page < C::kVK ? page : C::kVK);
  if (e != cudaSuccess) return e;
  static OnEveryDevice ready;
  e = ready([] {
    return attn_prepare_kernel(attn_tiles_kernel<NS>, C::kSmem, C::kThreads, C::kNQ == 2 ? 104 * 128 + 200 * 256 : 0);
  });
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
  return cudaLaunchKernelEx(&cfg, attn_tiles_kernel<NS>, mq, mk, mv, a);
}

cudaError_t launch_attn_tiles(const AttnArgs& a, cudaStream_t s) {
  switch ((a.dim + 63) / 64) {
    case 1: return launch_tiles<1>(a, s);
    case 2: return launch_tiles<2>(a, s);
    case 3: return launch_tiles<3>(a, s);
    default: return launch_tiles<4>(a, s);
  }
}

size_t attn_tiles_work_bytes(int dim) { return attn_work_bytes(kAttnCtas, dim <= 128 ? 256 : 128, dim); }

}  // namespace gsi
