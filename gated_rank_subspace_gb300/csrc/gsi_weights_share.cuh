// How the work of gathering attention weights over ragged requests is cut into
// equal shares: integer arithmetic on the lengths.  (It stands by itself, so that
// a program without a GPU can run it.)
#pragma once

#include "gsi_kernels.h"

namespace gsi {

// For key j of a request under a key/value head, with the logarithm L of each
// query row's sum (the attention's):
//   w_j = sum over the request's tokens i that see j, and the head's query
//         heads, of exp(scale q_i . k_j - L_i).
// A sum over rows for each key, so the kernels hold keys and run through the
// rows: a unit is a tile of KT keys of one request under one key/value head, and
// its steps are the row tiles (tpt tokens of the G heads) that see a key of it.
// All units' steps, in the order of requests, heads and key tiles, form one
// line; CTA b of G takes the steps [S b / G, S (b + 1) / G) of it.
//
// tpt is a power of two that divides KT, so the row tiles that tile t loses to
// the causal mask are t k - c, with k = KT / tpt and c = ceil((len - q_len) /
// tpt): the steps of the first x tiles are an arithmetic series.
constexpr int kKwCtas = 304;  // CTAs of a launch, at most: two an SM

struct KwReq {
  int q0, q_len, len, held;
};
struct KwSeg {
  KwReq q;
  int r, h, t;       // request, head, key tile
  int u0, n, a, b;   // first row tile, steps of the unit, this part of them
  long long first;   // the unit's first step on the line
};

template <int KT>
struct KwShape {
  int tpt;   // tokens of a row tile, a power of two
  int shift; // its logarithm

  __device__ __forceinline__ KwReq request(const KeyWeightArgs& a, int r) const {
    const int s = __ldcg(a.q_start + r), e = __ldcg(a.q_start + r + 1), n = __ldcg(a.kv_len + r);
    KwReq q;
    q.q0 = min(max(s, 0), a.N);
    q.q_len = min(max(e, q.q0), a.N) - q.q0;
    q.len = min(max(n, 0), int(a.width << a.page_shift));
    q.held = a.held ? min(max(__ldcg(a.held + r), 0), q.len) : 0;
    return q;
  }
  __device__ __forceinline__ int tiles(const KwReq& q) const { return int((q.len + int64_t(KT) - 1) / KT); }
  // the tiles that are visited: without tokens only those of keys that have to be begun at zero
  __device__ __forceinline__ int first_tile(const KwReq& q) const {
    return q.q_len > 0 ? 0 : q.held >= q.len ? tiles(q) : q.held / KT;
  }
  __device__ __forceinline__ int row_tiles(const KwReq& q) const { return (q.q_len + tpt - 1) >> shift; }
  // c above; without a mask no tile loses any
  __device__ __forceinline__ long long skip(const KeyWeightArgs& a, const KwReq& q) const {
    return a.causal ? -(-(long long)(q.len - q.q_len) >> shift) : (1ll << 40);
  }
  // first row tile that sees a key of tile t, and how many do (one step at least)
  __device__ __forceinline__ void steps(const KeyWeightArgs& a, const KwReq& q, int t, int& u0, int& n) const {
    const long long u = (long long)t * (KT >> shift) - skip(a, q);
    u0 = u > 0 ? int(u) : 0;
    n = max(1, row_tiles(q) - u0);
  }
  // steps of the tiles before x
  __device__ __forceinline__ long long prefix(const KeyWeightArgs& a, const KwReq& q, int x) const {
    const int t0 = first_tile(q);
    if (q.q_len == 0) return max(0, x - t0);
    const long long k = KT >> shift, c = skip(a, q), nq = row_tiles(q);
    const long long full = c >= 0 ? c / k + 1 : 0, z = full < x ? full : x;
    return z * nq + (x - z) * (nq + c) - k * ((long long)x * (x - 1) - z * (z - 1)) / 2;
  }
  __device__ __forceinline__ long long head_steps(const KeyWeightArgs& a, const KwReq& q) const {
    return q.len > 0 ? prefix(a, q, tiles(q)) : 0;
  }
};

// A CTA's share, walked part by part; every role of a CTA walks it alike.
template <int KT>
struct KwWalk {
  KwShape<KT> shape;
  KwReq q;
  int r, h, t;
  long long off;              // steps of the tile at t that lie before this place
  long long total, pos, end;  // steps of the line, and this CTA's
  int grid;                   // CTAs that have a share

  __device__ __forceinline__ bool next(const KeyWeightArgs& a, KwSeg& g) {
    if (pos >= end) return false;
    while (t >= shape.tiles(q)) {  // the next head or request with a step (there is one)
      if (q.len > shape.first_tile(q) * KT && h + 1 < a.hkv) {
        ++h;
      } else {
        q = shape.request(a, ++r);
        h = 0;
      }
      t = shape.first_tile(q);
    }
    shape.steps(a, q, t, g.u0, g.n);
    g.q = q;
    g.r = r;
    g.h = h;
    g.t = t;
    g.first = pos - off;
    const long long left = end - pos;
    g.a = int(off);
    g.b = g.n - off < left ? g.n : int(off + left);
    pos += g.b - g.a;
    off = 0;
    ++t;
    return true;
  }
  // The CTAs that hold parts of a unit.
  __device__ __forceinline__ void parts(const KwSeg& g, int& b0, int& b1) const {
    b0 = int(((g.first + 1) * grid + total - 1) / total) - 1;
    b1 = int(((g.first + g.n) * grid - 1) / total);
  }
};

// The share of CTA blockIdx.x; all NT threads of the block.
template <int KT, int NT>
__device__ __forceinline__ void kw_share(const KeyWeightArgs& a, int tpt, KwWalk<KT>& w) {
  __shared__ long long s_sum[NT / 32];
  __shared__ KwWalk<KT> s_walk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  KwShape<KT> shape;
  shape.tpt = tpt;
  shape.shift = __ffs(tpt) - 1;
  const int r0 = int((long long)a.n_req * tid / NT), r1 = int((long long)a.n_req * (tid + 1) / NT);
  long long mine = 0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) mine += shape.head_steps(a, shape.request(a, r)) * a.hkv;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  long long total = 0, before = inc - mine;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    if (i < warp) before += s_sum[i];
    total += s_sum[i];
  }
  const int grid = int(total < (long long)gridDim.x ? total : (long long)gridDim.x);
  const bool some = int(blockIdx.x) < grid;
  const long long pos = some ? total * blockIdx.x / grid : 0, end = some ? total * (blockIdx.x + 1) / grid : 0;
  if (!some && tid == 0) {
    s_walk.pos = s_walk.end = 0;
  } else if (some && before <= pos && pos < before + mine) {
    KwWalk<KT> p;
    p.shape = shape;
    p.total = total;
    p.pos = pos;
    p.end = end;
    p.grid = grid;
    long long at = pos - before, per;
    p.r = r0;
#pragma unroll 1
    for (;; ++p.r) {
      p.q = shape.request(a, p.r);
      per = shape.head_steps(a, p.q);
      if (at < per * a.hkv) break;
      at -= per * a.hkv;
    }
    p.h = int(at / per);
    at -= p.h * per;
    int lo = shape.first_tile(p.q), hi = shape.tiles(p.q);  // the last tile that begins at or before `at`
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (shape.prefix(a, p.q, mid) <= at) lo = mid; else hi = mid;
    }
    p.t = lo;
    p.off = at - shape.prefix(a, p.q, lo);
    s_walk = p;
  }
  __syncthreads();
  w = s_walk;
}

}  // namespace gsi
