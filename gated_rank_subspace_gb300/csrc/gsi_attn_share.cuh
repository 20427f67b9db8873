// How the work of an attention over ragged requests is cut into equal shares:
// integer arithmetic on the lengths, the same in every kernel.  (It stands by
// itself, so that a program without a GPU can run it.)
#pragma once

#include "gsi_kernels.h"

namespace gsi {

constexpr int kAttnCtas = 152;  // CTAs of a launch, at most: one an SM (two over a float32 cache)

// ------------------------------------------------------------------ work
// A unit is a block of `ut` consecutive new tokens of one request under one
// key/value head (their ut * group query rows), over the tiles of `kt` keys
// that any of its rows sees.  All units' tiles, in the order of requests,
// heads and token blocks, form one line; CTA b of G takes the tiles
// [T b / G, T (b + 1) / G) of it.  So the shares are equal to a tile whatever
// the lengths are, one long request is spread over all CTAs, and neighbours
// read the same keys.  A unit that sees no key counts as one tile (its rows
// of zeros have to be written).  Each CTA finds its share from the lengths.
// Where the shares are long enough for it, a unit counts for `extra` tiles
// more than it has (before its first one: what it costs to begin and to
// finish it), and a cut that falls within `extra` of a unit's end is moved
// there, since a part of a unit costs about that much to write and join.
struct AttnReq {
  int q0, q_len, len;
};

__device__ __forceinline__ AttnReq attn_request(const AttnArgs& a, int r) {
  const int s = __ldcg(a.q_start + r), e = __ldcg(a.q_start + r + 1), n = __ldcg(a.kv_len + r);
  AttnReq q;
  q.q0 = min(max(s, 0), a.N);
  q.q_len = min(max(e, q.q0), a.N) - q.q0;
  q.len = min(max(n, 0), int(a.width << a.page_shift));
  return q;
}

// The keys [lo, lim) that token i of a request sees.
__device__ __forceinline__ int attn_lim(const AttnArgs& a, const AttnReq& q, int i) {
  return a.causal ? max(0, q.len - q.q_len + i + 1) : q.len;
}
__device__ __forceinline__ int attn_lo(const AttnArgs& a, int lim) {
  return a.window > 0 && lim > a.window ? lim - a.window : 0;
}

// First tile and number of tiles of unit u.
__device__ __forceinline__ void attn_tiles(const AttnArgs& a, const AttnReq& q, int u, int ut, int kt, int& t0, int& n) {
  const int lim = attn_lim(a, q, min((u + 1) * ut, q.q_len) - 1);
  t0 = attn_lo(a, attn_lim(a, q, u * ut)) / kt;
  n = max(0, (lim + kt - 1) / kt - t0);
}

// Whole quotient of a by b > 0 (in 32 bits, a fifth of the time, where they suffice).
__device__ __forceinline__ long long attn_div(long long a, long long b) {
  if (((a | b) >> 31) == 0) return int(a) / int(b);
  return a / b;
}

// sum of floor((x i + y) / m) for i = 0 .. n - 1; x > 0, y >= 0, m a power of
// two.  Where x is one too (as many heads a group) in a few steps, else by
// Euclid's algorithm on x and m.
__device__ __forceinline__ long long attn_floor_sum(long long n, int m_, int x_, long long y) {
  if ((x_ & (x_ - 1)) == 0) {
    const int ms = __ffs(m_) - 1, xs = __ffs(x_) - 1;
    if (xs >= ms) return n * (y >> ms) + ((n * (n - 1) / 2) << (xs - ms));
    // floor((i + z) / 2^d) from z on
    const int d = ms - xs;
    const long long z = y >> xs, a = (n + z) >> d, b = z >> d;
    return ((a * (a - 1) / 2) << d) + a * (n + z - (a << d)) - ((b * (b - 1) / 2) << d) - b * (z - (b << d));
  }
  long long s = 0, m = m_, x = x_;
  while (n > 0) {
    if (x >= m) {
      const long long q = attn_div(x, m);
      s += (n - 1) * n / 2 * q;
      x -= q * m;
    }
    if (y >= m) {
      const long long q = attn_div(y, m);
      s += n * q;
      y -= q * m;
    }
    const long long top = x * n + y;
    if (top < m) break;
    n = attn_div(top, m);
    y = top - n * m;
    const long long z = m;
    m = x;
    x = z;
  }
  return s;
}

// Tiles of the first u units (all of them whole) of a request under one head.
// Two are counted one by one (~200 cycles each, a chain of dependent integer
// steps); more in closed form: unit v ends at the limit base + (v + 1) ut of its
// last token, and begins, under a window, window - 1 keys before that of its
// first.  (Not inlined: this runs once a CTA, and then its time is that of
// fetching its instructions.)
constexpr int kAttnCount = 2;
static __device__ __noinline__ long long attn_prefix_tiles(const AttnArgs& a, AttnReq q, int u, int ut, int kt) {
  const long long n = u;
  if (u <= kAttnCount) {
    int tiles = 0;
#pragma unroll 1
    for (int v = 0; v < u; ++v) {
      int t0, c;
      attn_tiles(a, q, v, ut, kt, t0, c);
      tiles += max(1, c);
    }
    return tiles;
  }
  if (!a.causal) return n * max(1, (q.len + kt - 1) / kt);
  const long long base = q.len - q.q_len;
  const long long none = base < 0 ? min(n, attn_div(-base, ut)) : 0;  // units that see no key
  long long s = none + attn_floor_sum(n - none, kt, ut, base + (none + 1) * ut + kt - 1);
  if (a.window > 0) {
    const long long first = base + 1 - a.window;  // where unit 0 begins
    const long long skip = first < 0 ? min(n, attn_div(-first + ut - 1, ut)) : 0;
    s -= attn_floor_sum(n - skip, kt, ut, first + skip * ut);
  }
  return s;
}

__device__ __forceinline__ int attn_units(const AttnReq& q, int ut) { return q.q_len > 0 ? (q.q_len - 1) / ut + 1 : 0; }

// Tiles of all units of a request under one head.
__device__ __forceinline__ long long attn_head_tiles(const AttnArgs& a, const AttnReq& q, int ut, int kt) {
  const int units = attn_units(q, ut);
  if (units == 0) return 0;
  int t0, n;
  attn_tiles(a, q, units - 1, ut, kt, t0, n);  // the last unit may be a part of one
  return (units > 1 ? attn_prefix_tiles(a, q, units - 1, ut, kt) : 0) + max(1, n);
}

// A place on the line: `off` tiles into unit u of head h of request r.
struct AttnPlace {
  AttnReq q;
  int r, h, u;
  long long off;
  // the beginning of the first request from r_ on that has tokens (there is one)
  __device__ __forceinline__ void start(const AttnArgs& a, int r_) {
    for (r = r_;; ++r) {
      q = attn_request(a, r);
      if (q.q_len > 0) break;
    }
    h = u = 0;
    off = 0;
  }
  // `at` tiles behind the first one of request r, whose lengths are q (there are tiles beyond); the 32 lanes of a warp,
  // alike: each counts a unit
  __device__ __noinline__ void set(const AttnArgs& a, int r_, AttnReq q_, long long at, int ut, int kt, int extra) {
    const int lane = threadIdx.x & 31;
    r = r_;
    q = q_;
    long long per_head;
#pragma unroll 1
    for (;;) {
      per_head = attn_head_tiles(a, q, ut, kt) + (long long)extra * attn_units(q, ut);
      if (at < per_head * a.hkv) break;
      at -= per_head * a.hkv;
      q = attn_request(a, ++r);
    }
    h = int(attn_div(at, per_head));
    off = at - h * per_head;
    // the last unit that begins at or before `off`: by bisection to a warp's units, then a lane each
    const int units = attn_units(q, ut);
    int past = units;
    long long before = 0;
    u = 0;
#pragma unroll 1
    while (past - u > 32) {
      const int mid = (u + past) >> 1;
      const long long c = attn_prefix_tiles(a, q, mid, ut, kt) + (long long)extra * mid;
      if (c <= off) {
        u = mid;
        before = c;
      } else {
        past = mid;
      }
    }
    off -= before;
    int t0, n = 0, c = 0;
    if (u + lane < units) {
      attn_tiles(a, q, u + lane, ut, kt, t0, n);
      c = max(1, n) + extra;
    }
    long long inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int skip = __popc(__ballot_sync(0xffffffffu, u + lane < units && inc <= off));
    if (skip > 0) off -= __shfl_sync(0xffffffffu, inc, skip - 1);
    u += skip;
  }
  // the beginning of the next unit (there is one)
  __device__ __forceinline__ void next_unit(const AttnArgs& a, int ut) {
    off = 0;
    if ((u + 1) * ut < q.q_len) {
      ++u;
    } else if (h + 1 < a.hkv) {
      u = 0;
      ++h;
    } else {
      start(a, r + 1);
    }
  }
  // tiles by which a cut here is moved
  __device__ __forceinline__ int snap(const AttnArgs& a, int ut, int kt, int extra) const {
    int t0, n;
    attn_tiles(a, q, u, ut, kt, t0, n);
    const int c = max(1, n) + extra, rem = int(off);
    return rem <= extra ? -rem : c - rem <= extra ? c - rem : 0;
  }
};

struct AttnShare {
  long long total, pos, end;  // tiles of the line: all, and this CTA's
  int grid, extra;            // grid: the CTAs that have a share (all, or as many as there are tiles)
  int dealt;                  // units dealt out whole instead (their number)
};

// One causal request alone has units that shrink with their place.  They are
// dealt out whole, the longest first, back and forth over the CTAs, where the
// longest hand is at most what the line's cuts cost (kAttnCut tiles, and an
// eighth: parts are written, read and folded) above the mean: no unit is cut
// then.  2048 tokens of 16 x 256 (16 tiles at most, 14.3 the mean): 42 us, on the
// line 52; 4096 of 40 x 128 (90, 80) 159, on the line 176; 8192 of 32 x 128 401, on
// the line 429, of 16 x 256 422 and 448, but of 32 x 64 364 and 356; 1000 behind
// 4000 of 40 x 128 (73, 39), left on the line, 91, dealt out 122.
constexpr int kAttnCut = 5, kAttnDealRows = 16;
__device__ __forceinline__ int attn_dealt(int k, int cta, int n_cta) {  // a hand's k-th unit
  return k * n_cta + (k & 1 ? n_cta - 1 - cta : cta);
}

// The share of CTA blockIdx.x and where it begins; all NT threads of the block.
// Each half of the block goes over the requests, and finds one of the two cuts.
template <int NT>
__device__ __forceinline__ AttnShare attn_share(const AttnArgs& a, int ut, int kt, int extra, AttnPlace& begin) {
  constexpr int NH = NT / 2, NW = NH / 32;
  static_assert(NT % 64 == 0 && NT >= kAttnCtas, "halves of whole warps; a thread a CTA");
  __shared__ long long s_tiles[2 * NW], s_units[2 * NW], s_cut[2];
  __shared__ AttnPlace s_begin;
  const int tid = threadIdx.x, lane = tid & 31, half = tid / NH, warp = (tid >> 5) - half * NW;
  const int ht = tid - half * NH;
  const int r0 = int((long long)a.n_req * ht / NH), r1 = int((long long)a.n_req * (ht + 1) / NH);
  long long tiles = 0, units = 0;
  AttnReq q{};  // of request r0
#pragma unroll 1
  for (int r = r1 - 1; r >= r0; --r) {
    q = attn_request(a, r);
    tiles += attn_head_tiles(a, q, ut, kt) * a.hkv;
    units += (long long)attn_units(q, ut) * a.hkv;
  }
  long long it = tiles, iu = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, it, o), y = __shfl_up_sync(0xffffffffu, iu, o);
    if (lane >= o) it += x, iu += y;
  }
  if (lane == 31) {
    s_tiles[half * NW + warp] = it;
    s_units[half * NW + warp] = iu;
  }
  __syncthreads();
  it -= tiles;
  iu -= units;
  long long total = 0, total_units = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) it += s_tiles[half * NW + w], iu += s_units[half * NW + w];
    total += s_tiles[w];
    total_units += s_units[w];
  }
  AttnShare s;
  s.extra = total >= 4ll * extra * gridDim.x ? extra : 0;  // shares of fewer than 4 extra tiles are cut where they fall
  total += s.extra * total_units;
  const long long before = it + s.extra * iu, mine = tiles + s.extra * units;
  s.total = total;
  s.grid = int(total < (long long)gridDim.x ? total : (long long)gridDim.x);
  if (total > s.grid && total < 16 * s.grid) {
    // As few CTAs as leave the longest share as it is (512 tiles are 4 for 128 CTAs and for 152): fewer parts to join, and
    // shares that often end where units do.  Without and with, us: one token over 2048 keys of 16 x 256 17.4 and 14.6, over
    // 3000 of 16 x 128 20.0 and 13.9, 5000 21.4 and 15.5, 2500 of 40 x 128 24.5 and 21.5, 8000 of 32 x 128 35.3 and 34.2;
    // 128 tokens over 4000 keys of 8 x 256 79 and 69; float32, 100 of 900 keys, 2 requests of 8 / 4 x 128 63.7 and 61.8.
    // But 10,000 keys of 8 x 64 14.2 and 16.7, 20,000 16.5 and 19.0, and 200 tokens of 1500 keys, 2 requests of 32 / 8 x
    // 128, 33.5 and 40.3 (row tiles' parts that all end at once are not there when the first one looks for them).  From 16
    // tiles a share on the longest is within a sixteenth of the mean.
    const unsigned tiles = unsigned(total), most = (tiles + s.grid - 1) / unsigned(s.grid);
    s.grid = int((tiles + most - 1) / most);
  }
  s.pos = s.end = 0;
  s.dealt = 0;
  if (extra > 0 && a.n_req == 1 && a.causal && a.window == 0 && total_units >= gridDim.x && total_units < (1ll << 30)) {
    const AttnReq all = attn_request(a, 0);
    const int n_units = int(total_units), n_cta = int(gridDim.x), rows = (n_units + n_cta - 1) / n_cta;
    bool deal;
    if (rows > kAttnDealRows) {
      deal = all.len == all.q_len;  // a whole prompt's last rows are its shortest units
    } else {
      int load = 0;  // of CTA tid
      if (tid < n_cta)
#pragma unroll 1
        for (int k = 0; k < rows; ++k) {
          const int i = attn_dealt(k, tid, n_cta);
          if (i < n_units) {
            int t0, n;
            attn_tiles(a, all, attn_units(all, ut) - 1 - i / a.hkv, ut, kt, t0, n);
            load += max(1, n) + s.extra;
          }
        }
      deal = !__syncthreads_or((long long)(load - kAttnCut) * n_cta * 8 > total * 9);
    }
    if (deal) {
      s.dealt = n_units;
      begin.q = all;
      begin.r = begin.h = begin.u = 0;
      begin.off = 0;  // units taken
      return s;
    }
  }
  const bool some = int(blockIdx.x) < s.grid;
  if (some) {
    const long long cut = attn_div(total * (blockIdx.x + half), s.grid);
    const unsigned hit = __ballot_sync(0xffffffffu, before <= cut && cut < before + mine);
    if (hit && (half == 0 || s.extra > 0)) {
      const int from = __ffs(hit) - 1;
      q.q0 = __shfl_sync(0xffffffffu, q.q0, from);
      q.q_len = __shfl_sync(0xffffffffu, q.q_len, from);
      q.len = __shfl_sync(0xffffffffu, q.len, from);
      AttnPlace p;
      p.set(a, __shfl_sync(0xffffffffu, r0, from), q, __shfl_sync(0xffffffffu, cut - before, from), ut, kt, s.extra);
      const int move = s.extra > 0 ? p.snap(a, ut, kt, s.extra) : 0;
      if (half == 0) {
        if (move > 0 && cut + move < total) p.next_unit(a, ut);
        if (move < 0) p.off += move;
        if (lane == 0) s_begin = p;
      }
      if (lane == 0) s_cut[half] = cut + move;
    } else if (hit && lane == 0) {
      s_cut[half] = cut;
    }
  }
  __syncthreads();
  if (some) {
    s.pos = s_cut[0];
    s.end = int(blockIdx.x) + 1 == s.grid ? total : s_cut[1];
    begin = s_begin;
  }
  return s;
}

// One part of a unit: its tiles [a, b) of n.
struct AttnSeg {
  AttnReq q;
  int r, h, u;
  int t0, n, a, b;
  long long first, last;  // the unit's place on the line
};

// Walks a share segment by segment; every role of a CTA walks it alike.
struct AttnWalk {
  AttnShare s;
  int ut, kt;
  AttnPlace p;

  __device__ __forceinline__ bool next(const AttnArgs& a, AttnSeg& g) {
    if (s.dealt > 0) {
      const int i = attn_dealt(int(p.off), int(blockIdx.x), int(gridDim.x));
      if (i >= s.dealt) return false;
      ++p.off;
      g.q = p.q;
      g.r = 0;
      g.u = attn_units(p.q, ut) - 1 - i / a.hkv;
      g.h = i % a.hkv;
      attn_tiles(a, p.q, g.u, ut, kt, g.t0, g.n);
      g.a = 0;
      g.b = g.n;
      g.first = 0;
      g.last = 1;
      return true;
    }
    if (s.pos >= s.end) return false;
    attn_tiles(a, p.q, p.u, ut, kt, g.t0, g.n);
    const long long cost = max(1, g.n) + s.extra;
    const long long take = cost - p.off < s.end - s.pos ? cost - p.off : s.end - s.pos;
    g.q = p.q;
    g.r = p.r;
    g.h = p.h;
    g.u = p.u;
    g.first = s.pos - p.off;
    g.last = g.first + cost;
    g.a = max(0, int(p.off) - s.extra);
    g.b = min(g.n, max(0, int(p.off + take) - s.extra));
    s.pos += take;
    p.off += take;
    if (p.off == cost && s.pos < s.end) p.next_unit(a, ut);
    return true;
  }
  // The CTAs that hold parts of a unit: the cuts inside it, beyond what is moved to its ends, are those of the CTAs
  // b0 + 1 .. b1 (none: b0 >= b1).
  __device__ __forceinline__ void parts(const AttnSeg& g, int& b0, int& b1) const {
    b0 = int(attn_div((g.first + s.extra + 1) * s.grid + s.total - 1, s.total)) - 1;
    b1 = int(attn_div((g.last - s.extra) * s.grid - 1, s.total));
  }
};

}  // namespace gsi
