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
// tpt): the steps of the first x tiles are an arithmetic series.  (A unit that no
// row sees counts as one step: its keys may have to begin at zero.)
constexpr int kKwCtas = 608;  // CTAs of a launch, at most: four an SM

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

// A CTA's share, walked part by part; every role of a CTA walks it alike, and few of its steps are more than additions.
template <int KT>
struct KwWalk {
  KwShape<KT> shape;
  KwReq q;
  int r, h, t;                // request, head, tile
  int first, tiles, row_tiles;
  long long u;                // first row tile that sees the tile, where positive
  long long off;              // steps of the tile at t that lie before this place
  long long total, pos, end;  // steps of the line, and this CTA's
  int grid;                   // CTAs that have a share

  __device__ __forceinline__ void enter(const KeyWeightArgs& a, const KwReq& q_, int t_) {  // tile t of a request
    q = q_;
    first = shape.first_tile(q);
    tiles = shape.tiles(q);
    row_tiles = shape.row_tiles(q);
    t = t_ < 0 ? first : t_;
    u = (long long)t * (KT >> shape.shift) - shape.skip(a, q);
  }
  __device__ __forceinline__ bool next(const KeyWeightArgs& a, KwSeg& g) {
    if (pos >= end) return false;
    while (t >= tiles) {  // the next head or request with a step (there is one)
      if (tiles > first && h + 1 < a.hkv) {
        ++h;
        enter(a, q, -1);
      } else {
        h = 0;
        enter(a, shape.request(a, ++r), -1);
      }
    }
    g.u0 = u > 0 ? int(u) : 0;
    g.n = max(1, row_tiles - g.u0);
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
    u += KT >> shape.shift;
    return true;
  }
  // The CTAs that hold parts of a unit.
  __device__ __forceinline__ void parts(const KwSeg& g, int& b0, int& b1) const {
    b0 = int(((g.first + 1) * grid + total - 1) / total) - 1;
    b1 = int(((g.first + g.n) * grid - 1) / total);
  }
};

// Whole quotient of a by b > 0 (in 32 bits, a fifth of the time, where they suffice).
__device__ __forceinline__ long long kw_div(long long a, long long b) {
  if (((a | b) >> 31) == 0) return int(a) / int(b);
  return a / b;
}

// The share of CTA blockIdx.x; all NT threads of the block.
template <int KT, int NT>
__device__ __forceinline__ void kw_share(const KeyWeightArgs& a, int tpt, KwWalk<KT>& w) {
  __shared__ long long s_sum[NT / 32], s_at;
  __shared__ KwReq s_req;
  __shared__ int s_r;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  w.shape.tpt = tpt;
  w.shape.shift = __ffs(tpt) - 1;
  const int r0 = int((long long)a.n_req * tid / NT), r1 = int((long long)a.n_req * (tid + 1) / NT);
  long long mine = 0;
  KwReq q{};  // of request r0
#pragma unroll 1
  for (int r = r1 - 1; r >= r0; --r) {
    q = w.shape.request(a, r);
    mine += w.shape.head_steps(a, q) * a.hkv;
  }
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
  w.total = total;
  w.grid = int(total < (long long)gridDim.x ? total : (long long)gridDim.x);
  const bool some = int(blockIdx.x) < w.grid;
  w.pos = some ? kw_div(total * blockIdx.x, w.grid) : 0;
  w.end = some ? kw_div(total * (blockIdx.x + 1), w.grid) : 0;
  if (some && before <= w.pos && w.pos < before + mine) {  // the request, by the thread that counted it
    long long at = w.pos - before;
    int r = r0;
#pragma unroll 1
    for (;;) {
      const long long n = w.shape.head_steps(a, q) * a.hkv;
      if (at < n) break;
      at -= n;
      q = w.shape.request(a, ++r);
    }
    s_at = at;
    s_req = q;
    s_r = r;
  }
  __syncthreads();
  if (!some) return;
  // the head, and the last tile that begins at or before the place: a warp tries 32 at a time (each warp for itself)
  const KwReq mine_q = s_req;
  const long long per = w.shape.head_steps(a, mine_q);
  w.r = s_r;
  w.h = int(kw_div(s_at, per));
  const long long at = s_at - w.h * per;
  int lo = w.shape.first_tile(mine_q), hi = w.shape.tiles(mine_q);
#pragma unroll 1
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const long long mid = lo + (long long)(lane + 1) * step;
    const bool reached = mid < hi && w.shape.prefix(a, mine_q, int(mid)) <= at;
    lo += __popc(__ballot_sync(0xffffffffu, reached)) * step;
    hi = min(hi, lo + step);
  }
  w.enter(a, mine_q, lo);
  w.off = at - w.shape.prefix(a, mine_q, lo);
}

}  // namespace gsi
