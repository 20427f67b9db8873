// Eviction from a paged cache by accumulated weight.

#include "gsi_common.cuh"
#include "gsi_kernels.h"

namespace gsi {

// Of the n keys that request r holds under head h, B stay: the recent ones
// (place >= n + evicted so far - recent), then the first ones (place < sinks),
// then those of the largest weight, ties to the lowest index.  The kept keys at
// B .. n - 1 move, in order, into the gaps below B, in order: a mover's source
// never is another one's destination, and what does not have to move does not.
//
// A cluster takes one (request, head), a CTA of it a stretch of the keys, a warp a
// stretch of that:
//   1. each key's rank as a 32-bit whole number, kept in shared memory;
//   2. the B-th largest: three histograms over 11, 11 and 10 bits, added over the
//      cluster, each narrowing the number to one bin of the last;
//   3. per warp: how many equal it, then how many gaps and movers there are; the
//      warps' first numbers are sums over the warps and CTAs before;
//   4. the lists of gaps and movers (workspace), and the moves, dealt out to all
//      warps of the cluster: a pair a lane for addresses, weights and places, whole
//      rows by the warp.
// Bound by the bytes where much moves (a row of K and V read and written, 8 bytes
// a key), by the chain of steps at a decode step's one key.
constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32;
constexpr int kEvHeld = 16384;   // ranks in shared memory; more are formed again in every pass
constexpr int kEvBins = 2048, kEvMost = 8;
constexpr size_t kEvSmem = size_t(kEvHeld) * 4;

struct EvShared {
  int hist[kEvBins];             // read by the cluster
  int warps[3][kEvWarps];        // equal, gaps, movers
  int count[3];                  // of this CTA (read by the cluster)
  int found[2];                  // digit, rank within it
  int scan[kEvWarps];
};

// Whole numbers in the order of weights: NaN lowest, then -inf .. inf.
__device__ __forceinline__ uint32_t ev_rank(float w) {
  if (w != w) return 0;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 is 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kEvThreads, 2) cache_evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t ev_smem[];
  __shared__ EvShared sh;
  uint32_t* s_rank = ev_smem;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), c = int(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / C, r = unit / a.hkv, h = unit - r * a.hkv;
  pdl_launch_dependents();
  pdl_wait();
  const int n = int(min(int64_t(max(__ldcg(a.kv_len + r), 0)), a.width << a.page_shift));
  const int B = min(n, a.budget);
  const int gone = a.offsets ? __ldcg(a.offsets + r) : 0;
  if (h == 0 && c == 0 && tid == 0) {
    a.kept[r] = B;
    if (a.offsets_out) a.offsets_out[r] = gone + (n - B);
  }
  if (n == B) return;  // the whole cluster

  const int page = 1 << a.page_shift;
  const int32_t* table = a.table + int64_t(r) * a.width;
  auto mark = [&](int pg, int j) { return ((int64_t(pg) * a.hkv + h) << a.page_shift) + (j & (page - 1)); };
  const int64_t newest = int64_t(n) + gone - a.recent;
  auto rank_of = [&](int j) -> uint32_t {
    const int pg = __ldcg(table + (j >> a.page_shift));
    if (pg < 0 || pg >= a.n_pages) return 0;  // (no key: a place outside the cache goes first)
    const int64_t at = mark(pg, j);
    const float w = __ldcg(a.weight + at);
    const int place = __ldcg(a.place + at);
    return place >= newest ? 0xffffffffu : place < a.sinks ? 0xfffffffeu : ev_rank(w);
  };
  // this CTA's keys [j0, j1), this warp's [k0, k1)
  const int j0 = int(int64_t(n) * c / C), j1 = int(int64_t(n) * (c + 1) / C);
  const int k0 = j0 + int(int64_t(j1 - j0) * warp / kEvWarps), k1 = j0 + int(int64_t(j1 - j0) * (warp + 1) / kEvWarps);
  const bool held = j1 - j0 <= kEvHeld;
  auto rank = [&](int j) { return held ? s_rank[j - j0] : rank_of(j); };
  for (int e = tid; e < kEvBins; e += kEvThreads) sh.hist[e] = 0;
  if (held) {
#pragma unroll 4
    for (int j = j0 + tid; j < j1; j += kEvThreads) s_rank[j - j0] = rank_of(j);
  }
  __syncthreads();

  // ---- the B-th largest rank: `value`, of which the first `ties` stay
  uint32_t value = 0, mask = 0;
  int ties = B;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    for (int j = k0 + lane; j - lane < k1; j += 32) {
      const uint32_t x = j < k1 ? rank(j) : 0;
      const bool in = j < k1 && (x & mask) == value;
      const int bin = in ? int(x >> shift) & (bins - 1) : -1;
      const unsigned same = __match_any_sync(0xffffffffu, bin);  // one addition for all lanes of a bin
      if (in && lane == __ffs(same) - 1) atomicAdd(&sh.hist[bin], __popc(same));
    }
    cluster.sync();
    // a thread adds its neighbouring bins, from the top: bins 4 t .. 4 t + 3 of the reversed order
    int mine[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bin = bins - 1 - (tid * 4 + i);
      int v = 0;
      if (bin >= 0)
        for (int b = 0; b < C; ++b) v += cluster.map_shared_rank(sh.hist, b)[bin];
      mine[i] = v;
      sum += v;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sh.scan[warp] = inc;
    __syncthreads();
    int above = inc - sum;
    for (int w = 0; w < warp; ++w) above += sh.scan[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < ties && ties <= above + mine[i]) {
        sh.found[0] = bins - 1 - (tid * 4 + i);
        sh.found[1] = ties - above;
      }
      above += mine[i];
    }
    cluster.sync();  // the histograms have been read
    value |= uint32_t(sh.found[0]) << shift;
    mask |= uint32_t(bins - 1) << shift;
    ties = sh.found[1];
    for (int e = tid; e < kEvBins; e += kEvThreads) sh.hist[e] = 0;
    __syncthreads();
  }

  // ---- numbers of the warps' first equal key, gap and mover
  auto before = [&](int which) {  // of this warp: over the CTAs and warps before it; all warps have written theirs
    __syncthreads();
    if (tid == 0) {
      int s = 0;
      for (int w = 0; w < kEvWarps; ++w) s += sh.warps[which][w];
      sh.count[which] = s;
    }
    cluster.sync();
    int s = 0;
    for (int b = 0; b < c; ++b) s += cluster.map_shared_rank(sh.count, b)[which];
    for (int w = 0; w < warp; ++w) s += sh.warps[which][w];
    return s;
  };
  int eq = 0;
  for (int j = k0 + lane; j - lane < k1; j += 32) eq += __popc(__ballot_sync(0xffffffffu, j < k1 && rank(j) == value));
  if (lane == 0) sh.warps[0][warp] = eq;
  const int eq0 = before(0);
  // walks this warp's keys: f(j, there, stays)
  auto walk = [&](auto f) {
    int seen = eq0;
    for (int j = k0 + lane; j - lane < k1; j += 32) {
      const bool there = j < k1;
      const uint32_t x = there ? rank(j) : 0;
      const bool same = there && x == value;
      const unsigned b = __ballot_sync(0xffffffffu, same);
      const bool stays = there && (x > value || (same && seen + __popc(b & ((1u << lane) - 1u)) < ties));
      seen += __popc(b);
      f(j, there, stays);
    }
  };
  int gaps = 0, movers = 0;
  walk([&](int j, bool there, bool stays) {
    gaps += __popc(__ballot_sync(0xffffffffu, there && j < B && !stays));
    movers += __popc(__ballot_sync(0xffffffffu, there && j >= B && stays));
  });
  if (lane == 0) {
    sh.warps[1][warp] = gaps;
    sh.warps[2][warp] = movers;
  }
  int gap0 = before(1), mover0 = before(2);
  int32_t* list = a.moves + int64_t(unit) * 2 * a.budget;
  walk([&](int j, bool there, bool stays) {
    const bool gap = there && j < B && !stays, mover = there && j >= B && stays;
    const unsigned bg = __ballot_sync(0xffffffffu, gap), bm = __ballot_sync(0xffffffffu, mover);
    const unsigned below = (1u << lane) - 1u;
    if (gap) list[gap0 + __popc(bg & below)] = j;
    if (mover) list[a.budget + mover0 + __popc(bm & below)] = j;
    gap0 += __popc(bg);
    mover0 += __popc(bm);
  });
  int total = 0;
  for (int b = 0; b < C; ++b) total += cluster.map_shared_rank(sh.count, b)[1];
  __threadfence();
  cluster.sync();  // the lists are there, and no CTA's shared memory is read from here on

  // ---- the moves
  const int vec = a.row_bytes / 16;
  const int64_t head = h * a.head_stride;
  for (int i0 = (c * kEvWarps + warp) * 32; i0 < total; i0 += C * kEvThreads) {
    const int i = i0 + lane;
    long long from = -1, to = -1;
    if (i < total) {
      const int dj = __ldcg(list + i), sj = __ldcg(list + a.budget + i);
      const int dp = __ldcg(table + (dj >> a.page_shift)), sp = __ldcg(table + (sj >> a.page_shift));
      if (dp >= 0 && dp < a.n_pages && sp >= 0 && sp < a.n_pages) {
        from = (sp * a.page_stride + head + int64_t(sj & (page - 1)) * a.token_stride) * a.elem;
        to = (dp * a.page_stride + head + int64_t(dj & (page - 1)) * a.token_stride) * a.elem;
        const int64_t s = mark(sp, sj), d = mark(dp, dj);
        const float w = __ldcg(a.weight + s);
        const int p = __ldcg(a.place + s);
        a.weight[d] = w;
        a.place[d] = p;
      }
    }
    const int m = min(32, total - i0);
    // four pairs' rows in flight
    for (int p = 0; p < m; p += 4) {
      long long f[4], t[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        f[x] = __shfl_sync(0xffffffffu, from, p + x);
        t[x] = __shfl_sync(0xffffffffu, to, p + x);
      }
      for (int e = lane; e < 2 * vec; e += 32) {
        char* base = static_cast<char*>(e < vec ? a.K : a.V) + (e < vec ? e : e - vec) * 16;
        uint4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (f[x] >= 0) v[x] = ld_cg_v4(base + f[x]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (f[x] >= 0) *reinterpret_cast<uint4*>(base + t[x]) = v[x];
      }
    }
  }
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  static OnEveryDevice ready;
  const cudaError_t e =
      ready([] { return cudaFuncSetAttribute(cache_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kEvSmem)); });
  if (e != cudaSuccess) return e;
  const int64_t units = int64_t(a.n_req) * a.hkv, most = a.width << a.page_shift;
  unsigned C = 1;  // as many CTAs a unit as there are SMs for, of 512 keys at least
  while (C < unsigned(kEvMost) && units * C * 2 <= 2 * sm_count() && most > int64_t(C) * 512) C *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(units * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = kEvSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cache_evict_kernel, a);
}

}  // namespace gsi
