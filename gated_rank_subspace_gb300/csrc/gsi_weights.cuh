// Accumulated attention weights of cached keys: what their kernels share beside
// the shares of their work -- the sums of a unit that is cut, and a key's sum.
#pragma once

#include "gsi_async.cuh"
#include "gsi_weights_share.cuh"

namespace gsi {

// The parts of a unit that is cut: KT sums each, in the workspace.  The CTA
// that finds itself the last to arrive adds them in the order of the line (so
// the result does not depend on who came last) and sets the counter back to
// zero.  Nobody waits.  At most two units of a share are cut: one that an
// earlier CTA began (slot 2 b) and one that a later CTA ends (slot 2 b + 1).
// (The counters lie where the attention's do, the parts behind them: one workspace serves both.)
constexpr size_t kKwCounterBytes = 4096;
static_assert(4 * kKwCtas <= int(kKwCounterBytes), "a counter a CTA");
constexpr int kKwPart = 128;  // sums of a part, at most
inline size_t kw_work_bytes() { return sizeof(Ctrl) + kKwCounterBytes + size_t(2) * kKwCtas * kKwPart * 4; }
__device__ __forceinline__ unsigned* kw_counter(const KeyWeightArgs& a, int cta) {
  return reinterpret_cast<unsigned*>(static_cast<char*>(a.work) + sizeof(Ctrl)) + cta;
}
__device__ __forceinline__ float* kw_part(const KeyWeightArgs& a, int slot) {
  return reinterpret_cast<float*>(static_cast<char*>(a.work) + sizeof(Ctrl) + kKwCounterBytes) + size_t(slot) * kKwPart;
}
__device__ __forceinline__ uint32_t* kw_err(const KeyWeightArgs& a) { return &static_cast<Ctrl*>(a.work)->err; }

// Where a unit's key has its marks, and what it has gathered: two loads, one behind the other, that are issued before the sum
// is needed.
struct KwMark {
  int64_t at;  // none: -1
  float old;
  int shift;   // the request's offset
};
__device__ __forceinline__ KwMark kw_mark(const KeyWeightArgs& a, const KwSeg& g, int key) {
  KwMark m{-1, 0.f, 0};
  if (key >= g.q.len || (g.q.q_len == 0 && key < g.q.held)) return m;
  const int pg = __ldcg(a.table + int64_t(g.r) * a.width + (key >> a.page_shift));
  if (key >= g.q.held && a.offsets) m.shift = __ldcg(a.offsets + g.r);
  if (pg < 0 || pg >= a.n_pages) return m;
  m.at = ((int64_t(pg) * a.hkv + g.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
  if (key < g.q.held) m.old = __ldcg(a.weight + m.at);
  return m;
}
// Gives the sum of a unit's key to the key: added to what it has, or its first.  (The key has no other writer: a page belongs
// to one request.)
__device__ __forceinline__ void kw_give(const KeyWeightArgs& a, const KwSeg& g, int key, const KwMark& m, float sum) {
  if (m.at < 0) return;
  if (key < g.q.held) {
    a.weight[m.at] = m.old + sum;
  } else {
    a.weight[m.at] = sum;
    a.place[m.at] = key + m.shift;
  }
}

// A bf16 cache, on the tensor cores; few: steps of 16 query rows (else 128).  There is a row of Q, and a step holds a token's
// heads.
cudaError_t launch_key_weights_tiles(const KeyWeightArgs& a, bool few, cudaStream_t s);

}  // namespace gsi
