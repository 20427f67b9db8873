// What the attention kernels share: how the work of ragged requests is cut
// into equal shares, the partial results where a share ends inside a row
// tile, and the paged tensor maps.
#pragma once

#include <cuda.h>

#include "gsi_async.cuh"
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
// then.  2048 tokens of 16 x 256 (16 tiles at most, 14.3 the mean):
// 41 us, on the line 49; 4096 of 40 x 128 (90, 80) 162, on the line 175; 8192 of
// 32 x 128 394, on the line 417; but 1000 behind 4000 of 40 x 128 (73, 39) 133,
// on the line 93.
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
