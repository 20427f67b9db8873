// What the attention kernels share beside the shares of their work: the partial
// results where a share ends inside a row tile, and the paged tensor maps.
#pragma once

#include <cuda.h>

#include "gsi_async.cuh"
#include "gsi_attn_share.cuh"

namespace gsi {

// ------------------------------------------------------------------ partial results
// A unit that is cut has its parts in the shares of consecutive CTAs.  Each
// leaves its rows' running maximum m, sum l and unnormalised output o in the
// workspace; the CTA that finds itself the last to arrive at the unit's
// counter joins all parts in the order of the line (so the result does not
// depend on who came last) and sets the counter back to zero.  Nobody waits.
// At most two units of a share are cut: one that an earlier CTA began (slot
// 2 b) and one that a later CTA ends (slot 2 b + 1).
constexpr size_t kAttnCounterBytes = 4096;
static_assert(2 * kAttnCtas * 2 * 4 <= int(kAttnCounterBytes), "two counters (row tiles) a CTA");

__host__ __device__ constexpr size_t attn_slot_floats(int rows, int dim) { return size_t(rows) * (dim + 2); }
inline size_t attn_work_bytes(int ctas, int rows, int dim) {
  return (sizeof(Ctrl) + kAttnCounterBytes + 2 * size_t(ctas) * attn_slot_floats(rows, dim) * 4 + 255) / 256 * 256;
}
__device__ __forceinline__ uint32_t* attn_err(const AttnArgs& a) { return &static_cast<Ctrl*>(a.work)->err; }
__device__ __forceinline__ unsigned* attn_counter(const AttnArgs& a, int cta, int tile) {
  return reinterpret_cast<unsigned*>(static_cast<char*>(a.work) + sizeof(Ctrl)) + 2 * cta + tile;
}
// The part of row tile `tile` (of `tiles` of a unit, `rows` rows each) in a
// slot: m[rows], l[rows], then o in 16-byte pieces -- a row's pieces side by
// side (kRowMajor), or one piece of every row side by side, which is how
// threads that own a row each store them in whole lines.
__device__ __forceinline__ float* attn_part(const AttnArgs& a, int slot, int tiles, int tile, int rows) {
  return reinterpret_cast<float*>(static_cast<char*>(a.work) + sizeof(Ctrl) + kAttnCounterBytes) +
         (size_t(slot) * tiles + tile) * attn_slot_floats(rows, a.dim);
}
template <bool kRowMajor>
__device__ __forceinline__ float4* attn_piece(float* part, int rows, int dim, int row, int c) {
  return reinterpret_cast<float4*>(part + 2 * rows) + (kRowMajor ? row * (dim / 4) + c / 4 : (c / 4) * rows + row);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp2(m - to) for running maxima, where -inf stands for "no key yet".
__device__ __forceinline__ float attn_scale(float m, float to) { return m == -INFINITY ? 0.f : ex2(m - to); }

// Number of the output row of query row `row` (token-major, head-minor) of a
// row tile that begins with token tok0 of the request.
__device__ __forceinline__ int64_t attn_out_row(const AttnArgs& a, const AttnSeg& g, int tok0, int row) {
  const int tok = row / a.group;
  return (int64_t(g.q.q0 + tok0 + tok) * a.hkv + g.h) * a.group + (row - tok * a.group);
}

__device__ __forceinline__ uint32_t attn_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Eight finished values of an output row.
template <class T>
__device__ __forceinline__ void attn_store8(const AttnArgs& a, int64_t at, const float (&v)[8]) {
  if constexpr (T::kBytes == 2) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.O) + at) =
        make_uint4(attn_pack(v[0], v[1]), attn_pack(v[2], v[3]), attn_pack(v[4], v[5]), attn_pack(v[6], v[7]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.O) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Folds the parts from .. to of a row tile whose first part is b0's into the
// state (m, l, o[CW], from column c) of one row.  All loads of a part are in
// flight together.  Starting from the first part's own values or from nothing
// gives the same bits.
template <bool kRowMajor, int CW>
__device__ __forceinline__ void attn_fold(const AttnArgs& a, int from, int to, int b0, int tiles, int tile, int rows,
                                          int row, int c, float& m, float& l, float (&o)[CW]) {
#pragma unroll(CW <= 8 ? 8 : 1)
  for (int b = from; b <= to; ++b) {
    float* p = attn_part(a, 2 * b + (b == b0), tiles, tile, rows);
    const float mp = __ldcg(p + row), lp = __ldcg(p + rows + row);
    float4 v[CW / 4];
#pragma unroll
    for (int i = 0; i < CW / 4; ++i)
      v[i] = c + 4 * i < a.dim ? __ldcg(attn_piece<kRowMajor>(p, rows, a.dim, row, c + 4 * i)) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float mm = fmaxf(m, mp), f = attn_scale(m, mm), fp = attn_scale(mp, mm);
    m = mm;
    l = l * f + lp * fp;
#pragma unroll
    for (int i = 0; i < CW / 4; ++i) {
      o[4 * i] = fmaf(v[i].x, fp, o[4 * i] * f);
      o[4 * i + 1] = fmaf(v[i].y, fp, o[4 * i + 1] * f);
      o[4 * i + 2] = fmaf(v[i].z, fp, o[4 * i + 2] * f);
      o[4 * i + 3] = fmaf(v[i].w, fp, o[4 * i + 3] * f);
    }
  }
}

// 1 / l for a row of token tok.  A sum of 0 is that of a row without a key, whose output is zeros, or of one whose scores are
// all -inf, which has no softmax (any other row's largest weight is about 1).
__device__ __forceinline__ float attn_inverse(const AttnArgs& a, const AttnReq& q, int tok, float l) {
  if (l != 0.f) return 1.f / l;
  return attn_lim(a, q, tok) > 0 ? NAN : 0.f;
}

// Writes CW columns from c of a finished row of token tok: o / l.
template <class T, int CW>
__device__ __forceinline__ void attn_finish(const AttnArgs& a, const AttnReq& q, int tok, int64_t at, int c, float l,
                                            const float (&o)[CW]) {
  const float inv = attn_inverse(a, q, tok, l);
  if constexpr (CW == 4) {
    static_assert(T::kBytes == 4, "pieces of four are float32's");
    *reinterpret_cast<float4*>(static_cast<float*>(a.O) + at) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  } else if (CW >= 16 && T::kBytes == 2 && a.dim % 16 == 0 && (reinterpret_cast<uintptr_t>(a.O) & 31) == 0) {
    // whole sectors: a thread with a row of its own writes 32 bytes at a time
#pragma unroll
    for (int i = 0; i + 16 <= CW; i += 16) {
      uint32_t w[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) w[x] = attn_pack(o[i + 2 * x] * inv, o[i + 2 * x + 1] * inv);
      if (c + i < a.dim)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<uint16_t*>(a.O) + at + i),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    }
  } else {
#pragma unroll
    for (int i = 0; i < CW; i += 8) {
      float w[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) w[x] = o[i + x] * inv;
      if (c + i < a.dim) attn_store8<T>(a, at + i, w);
    }
  }
}

// Joins all parts of a row tile and writes its rows; threads tid of nt.
template <class T, bool kRowMajor, int CW>
__device__ __forceinline__ void attn_join(const AttnArgs& a, const AttnSeg& g, int b0, int b1, int tiles, int tile,
                                          int rows, int n_rows, int tok0, int tid, int nt) {
  const int per = (a.dim + CW - 1) / CW;
  for (int e = tid; e < n_rows * per; e += nt) {
    const int row = kRowMajor ? e / per : e % n_rows, c = (kRowMajor ? e % per : e / n_rows) * CW;
    float m = -INFINITY, l = 0.f, o[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) o[i] = 0.f;
    attn_fold<kRowMajor, CW>(a, b0, b1, b0, tiles, tile, rows, row, c, m, l, o);
    attn_finish<T, CW>(a, g.q, tok0 + row / a.group, attn_out_row(a, g, tok0, row) * a.dim + c, c, l, o);
  }
}

// The values that a masked tile hides from some rows are multiplied by
// weights of zero, which hides numbers but not infinities and NaN.  The
// kernels therefore take non-finite values out of such tiles, and where one
// was found (`found`) this adds it to the rows that do see its key: the sum
// with it is what the definition gives.  Tiles [t0 + a, t0 + b) of kt keys;
// the value of column c for a row that sees [lo, lim).
template <class T>
static __device__ __noinline__ float attn_nonfinite(const AttnArgs& a, const AttnSeg& g, int kt, int lo, int lim, int lo_all,
                                             int lim_all, int c, float o) {
  for (int t = g.t0 + g.a; t < g.t0 + g.b; ++t) {
    if (t * kt >= lo_all && (t + 1) * kt <= lim_all) continue;  // every row sees this tile: nothing was taken out
    for (int j = max(t * kt, lo); j < min((t + 1) * kt, lim); ++j) {
      const int64_t pg = __ldcg(a.table + int64_t(g.r) * a.width + (j >> a.page_shift));
      if (pg < 0 || pg >= a.n_pages) continue;
      const float v = T::load1_cg(a.V, pg * a.page_stride + g.h * a.head_stride +
                                           int64_t(j & ((1 << a.page_shift) - 1)) * a.token_stride + c);
      if (!(fabsf(v) < INFINITY)) o += v;
    }
  }
  return o;
}

// ------------------------------------------------------------------ paged tensor maps
// Box loads of a paged operand: coordinates (column, token of the page, head, page).
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, int tok, int head,
                                              int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(col), "r"(tok), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// Maps of K and V with boxes of 64 columns x box_rows tokens (128-byte
// swizzle; columns beyond head_dim and pages outside the cache read as zeros).
cudaError_t attn_page_map(CUtensorMap* m, const AttnArgs& a, const void* base, int box_rows);

// Shared memory for a kernel, and the registers its warpgroups trade: setmaxnreg.inc waits for what the launch's
// registers do not hold, so a build that gave the kernel fewer than `regs` a block is refused here.
template <class K>
inline cudaError_t attn_prepare_kernel(K kern, size_t smem, int threads, int regs) {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, kern);
  if (e != cudaSuccess) return e;
  if (at.numRegs * threads < regs) return cudaErrorInvalidKernelImage;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
}

// Map of the query rows: (column, head, token) boxes of 64 x box_heads x box_tokens.
cudaError_t attn_query_map(CUtensorMap* m, const AttnArgs& a, int box_heads, int box_tokens);

// Units of at most 8 query rows.
cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_tiles(const AttnArgs& a, cudaStream_t s);
// A float32 cache: units of 64 query rows (few: 16).
cudaError_t launch_attn_f32(const AttnArgs& a, bool few, cudaStream_t s);
size_t attn_tiles_work_bytes(int dim);

}  // namespace gsi
