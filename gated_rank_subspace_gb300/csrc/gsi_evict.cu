// Eviction from a paged cache by accumulated weight.

#include "gsi_async.cuh"
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
//   2. the B-th largest: four histograms of 8 bits, added over the cluster, each
//      narrowing the number to one bin of the last (wider ones cost more to add
//      than the pass they save: three of 11, 11 and 10 bits 28 us where four take
//      25, 80 heads of up to 8003 keys, nothing to move), until a bin stays whole;
//   3. per warp: how many equal it, then how many gaps and movers there are; the
//      warps' first numbers are sums over the warps and CTAs before;
//   4. the lists of gaps and movers (workspace), and the moves, dealt out to all
//      warps of the cluster.
// Few keys given up (a decode step's one) are found without histograms, as the
// lowest ranks one after the other, by one CTA.
// Bound by the bytes where much moves (a row of K and V read and written, 8 bytes
// a key: 80 heads of up to 8003 keys of 256 columns to 2048 59 us, of which 40 are
// moves at 5.3 TB/s), by the chain of steps at a decode step's one key (128 heads of 1025
// keys 6 us).
constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32;
// Ranks in a CTA's shared memory: 131,072 a head up to 57 heads (eight CTAs each), 16,384 from 229 on (one).  More are formed again
// in every pass (256 heads of 16,385 to 16,640 keys to 8192 304 us, of 16,384 228; one key of 16,385 99, of 16,384 23).
constexpr int kEvHeld = 16384;
constexpr int kEvBins = 256, kEvMost = 8;
constexpr int kEvBuf = 6144;     // bytes of a warp's rows in flight
constexpr int kEvFew = 8;        // keys given up that are found one by one
constexpr size_t kEvSmem = size_t(kEvHeld) * 4 > size_t(kEvWarps) * kEvBuf ? size_t(kEvHeld) * 4 : size_t(kEvWarps) * kEvBuf;
static_assert(kEvBuf >= 2 * 1024 && kEvBuf % 16 == 0, "two rows of 256 float32 values");

struct EvShared {
  int hist[2][kEvBins];          // of a pass and the next one (read by the cluster)
  int warps[3][kEvWarps];        // equal, gaps, movers
  int count[3];                  // of this CTA (read by the cluster)
  int found[3];                  // digit, rank within it, how many there are
  int scan[kEvWarps];
  unsigned long long low[kEvWarps];
  uint64_t bar[kEvWarps];        // a warp's rows in flight
  int gone[kEvFew], gap[kEvFew], mover[kEvFew];
  int n_moves;
};

// Whole numbers in the order of weights: NaN lowest, then -inf .. inf.
__device__ __forceinline__ uint32_t ev_rank(float w) {
  if (w != w) return 0;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 is 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kEvThreads, 2) cache_evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(128) uint32_t ev_smem[];
  __shared__ EvShared sh;
  uint32_t* s_rank = ev_smem;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), c = int(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / C, r = unit / a.hkv, h = unit - r * a.hkv;
  pdl_launch_dependents();
  if (tid < kEvWarps) bar_init(&sh.bar[tid], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
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
  const int vec = a.row_bytes / 16;
  const int64_t head = h * a.head_stride;
  auto row_of = [&](int pg, int j) { return (pg * a.page_stride + head + int64_t(j & (page - 1)) * a.token_stride) * a.elem; };
  // one key, by a warp
  auto move = [&](int dj, int sj) {
    const int dp = __ldcg(table + (dj >> a.page_shift)), sp = __ldcg(table + (sj >> a.page_shift));
    if (dp < 0 || dp >= a.n_pages || sp < 0 || sp >= a.n_pages) return;
    const int64_t from = row_of(sp, sj), to = row_of(dp, dj), s = mark(sp, sj), d = mark(dp, dj);
    for (int e = lane; e < 2 * vec; e += 32) {
      char* base = static_cast<char*>(e < vec ? a.K : a.V) + (e < vec ? e : e - vec) * 16;
      *reinterpret_cast<uint4*>(base + to) = ld_cg_v4(base + from);
    }
    if (lane == 0) a.weight[d] = __ldcg(a.weight + s);
    if (lane == 1) a.place[d] = __ldcg(a.place + s);
  };
  const int64_t newest = int64_t(n) + gone - a.recent;
  // ranks of the N keys from j on, `step` apart, those below `end`: their table entries, then their marks, in flight together
  auto ranks_of = [&](auto& out, int j, int step, int end) {
    constexpr int N = sizeof(out) / sizeof(out[0]);
    int pg[N], place[N];
    float w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) pg[i] = j + i * step < end ? __ldcg(table + ((j + i * step) >> a.page_shift)) : -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool there = pg[i] >= 0 && pg[i] < a.n_pages;
      const int64_t at = there ? mark(pg[i], j + i * step) : 0;
      w[i] = there ? __ldcg(a.weight + at) : 0.f;
      place[i] = there ? __ldcg(a.place + at) : 0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)  // (a place outside the cache has no key: the lowest)
      out[i] = pg[i] < 0 || pg[i] >= a.n_pages ? 0
               : place[i] >= newest            ? 0xffffffffu
               : place[i] < a.sinks            ? 0xfffffffeu
                                               : ev_rank(w[i]);
  };
  auto hold = [&](int from, int end) {  // the ranks of keys [from, end), which this CTA keeps
    for (int j = from + tid; j < end; j += 8 * kEvThreads) {
      uint32_t x[8];
      ranks_of(x, j, kEvThreads, end);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i * kEvThreads < end) s_rank[j - from + i * kEvThreads] = x[i];
    }
  };

  if (n - B <= kEvFew && n <= kEvHeld) {
    if (c != 0) return;
    hold(0, n);
    // the keys given up, from the lowest rank on; of equal ones the last first.  (A thread looks at the ranks it wrote.)
    unsigned long long last = 0;  // above the one found before
    for (int e = 0; e < n - B; ++e) {
      unsigned long long low = ~0ull;
      for (int j = tid; j < n; j += kEvThreads) {
        const unsigned long long x = (unsigned long long)s_rank[j] << 32 | (0xffffffffu - unsigned(j));
        if ((e == 0 || x > last) && x < low) low = x;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long x = __shfl_xor_sync(0xffffffffu, low, o);
        if (x < low) low = x;
      }
      __syncthreads();  // the warps' lowest before have been read
      if (lane == 0) sh.low[warp] = low;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kEvWarps; ++w) {
        const unsigned long long x = sh.low[w];
        if (x < low) low = x;
      }
      last = low;
      if (tid == 0) sh.gone[e] = int(0xffffffffu - unsigned(low));
    }
    __syncthreads();
    if (warp == 0) {
      const int mine = lane < n - B ? sh.gone[lane] : 0x7fffffff;  // a key given up
      const int next = B + lane;                                  // a key behind the new length
      int before = 0;
      bool stays = lane < n - B;
      for (int e = 0; e < n - B; ++e) {
        const int x = __shfl_sync(0xffffffffu, mine, e);
        before += x < mine;
        stays = stays && x != next;
      }
      if (mine < B) sh.gap[before] = mine;
      const unsigned b = __ballot_sync(0xffffffffu, stays);
      if (stays) sh.mover[__popc(b & ((1u << lane) - 1u))] = next;
      if (lane == 0) sh.n_moves = __popc(b);
    }
    __syncthreads();
    if (warp < sh.n_moves) move(sh.gap[warp], sh.mover[warp]);
    return;
  }

  // this CTA's keys [j0, j1), this warp's [k0, k1)
  const int j0 = int(int64_t(n) * c / C), j1 = int(int64_t(n) * (c + 1) / C);
  const int k0 = j0 + int(int64_t(j1 - j0) * warp / kEvWarps), k1 = j0 + int(int64_t(j1 - j0) * (warp + 1) / kEvWarps);
  const bool held = j1 - j0 <= kEvHeld;
  auto rank = [&](int j) {
    if (held) return s_rank[j - j0];
    uint32_t x[1];
    ranks_of(x, j, 1, k1);
    return x[0];
  };
  for (int e = tid; e < 2 * kEvBins; e += kEvThreads) (&sh.hist[0][0])[e] = 0;
  if (held) hold(j0, j1);
  __syncthreads();

  // ---- the B-th largest rank: `value`, of which the first `ties` stay
  uint32_t value = 0, mask = 0;
  int ties = B;
  bool all = false;  // every key of the bin stays: all ranks from `value` on
#pragma unroll 1
  for (int shift = 24, buf = 0; shift >= 0; shift -= 8, buf ^= 1) {
    for (int j = k0 + lane; j - lane < k1; j += 32) {
      const uint32_t x = j < k1 ? rank(j) : 0;
      const bool in = j < k1 && (x & mask) == value;
      const int bin = int(x >> shift) & (kEvBins - 1);
      const unsigned some = __ballot_sync(0xffffffffu, in);
      if (some == 0) continue;
      // one addition where all lanes have one bin (weights that are alike), else one each
      const int first = __ffs(some) - 1, theirs = __shfl_sync(0xffffffffu, bin, first);
      if (__all_sync(0xffffffffu, !in || bin == theirs)) {
        if (lane == first) atomicAdd(&sh.hist[buf][bin], __popc(some));
      } else if (in) {
        atomicAdd(&sh.hist[buf][bin], 1);
      }
    }
    cluster.sync();
    // bins from the top, a thread each
    const int bin = kEvBins - 1 - tid;
    int count = 0;
    if (bin >= 0) {
      for (int b = 0; b < C; ++b) count += cluster.map_shared_rank(sh.hist[buf], b)[bin];
      sh.hist[buf ^ 1][bin] = 0;  // (of the pass before: every CTA has read it)
    }
    int inc = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sh.scan[warp] = inc;
    __syncthreads();
    int above = inc - count;
    for (int w = 0; w < warp; ++w) above += sh.scan[w];
    if (above < ties && ties <= above + count) {  // one thread (those past the bins have no count)
      sh.found[0] = bin;
      sh.found[1] = ties - above;
      sh.found[2] = count;
    }
    __syncthreads();
    value |= uint32_t(sh.found[0]) << shift;
    mask |= uint32_t(kEvBins - 1) << shift;
    ties = sh.found[1];
    all = sh.found[2] == ties;
    if (all) break;
  }

  // ---- numbers of the warps' first equal key, gap and mover
  // sums over the CTAs and warps before this one, of the counts from `which` on; all warps have written theirs
  auto before = [&](int which, int n_counts, int* out) {
    __syncthreads();
    if (tid < n_counts) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < kEvWarps; ++w) s += sh.warps[which + tid][w];
      sh.count[which + tid] = s;
    }
    cluster.sync();
    for (int i = 0; i < n_counts; ++i) {
      int s = 0;
      for (int b = 0; b < c; ++b) s += cluster.map_shared_rank(sh.count, b)[which + i];
      for (int w = 0; w < warp; ++w) s += sh.warps[which + i][w];
      out[i] = s;
    }
  };
  int eq0 = 0;
  if (!all) {
    int eq = 0;
    for (int j = k0 + lane; j - lane < k1; j += 32) eq += __popc(__ballot_sync(0xffffffffu, j < k1 && rank(j) == value));
    if (lane == 0) sh.warps[0][warp] = eq;
    before(0, 1, &eq0);
  }
  // walks this warp's keys: f(j, there, stays)
  auto walk = [&](auto f) {
    int seen = eq0;
    for (int j = k0 + lane; j - lane < k1; j += 32) {
      const bool there = j < k1;
      const uint32_t x = there ? rank(j) : 0;
      const bool same = there && !all && x == value;
      const unsigned b = __ballot_sync(0xffffffffu, same);
      const bool stays = there && (same ? seen + __popc(b & ((1u << lane) - 1u)) < ties : x >= value);
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
  int at[2];
  before(1, 2, at);
  int gap0 = at[0], mover0 = at[1];
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
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ranks' memory becomes the rows'
  cluster.sync();  // the lists are there, and no CTA's shared memory is read from here on

  // ---- the moves: a warp's rows pass through its part of shared memory by bulk copies, a lane a row of K or V
  uint8_t* buf = reinterpret_cast<uint8_t*>(ev_smem) + warp * kEvBuf;
  const int pairs = min(32, kEvBuf / a.row_bytes) / 2, stride = C * kEvWarps * pairs;
  char* base = static_cast<char*>(lane & 1 ? a.V : a.K);
  struct Row {
    int64_t from, to, s, d;  // bytes of the row, marks; none: -1
  };
  auto row_at = [&](int i0) {
    const int i = i0 + (lane >> 1);
    if (lane < 2 * pairs && i < total) {
      const int dj = __ldcg(list + i), sj = __ldcg(list + a.budget + i);
      const int dp = __ldcg(table + (dj >> a.page_shift)), sp = __ldcg(table + (sj >> a.page_shift));
      if (dp >= 0 && dp < a.n_pages && sp >= 0 && sp < a.n_pages) return Row{row_of(sp, sj), row_of(dp, dj), mark(sp, sj), mark(dp, dj)};
    }
    return Row{-1, -1, -1, -1};
  };
  int i0 = (c * kEvWarps + warp) * pairs;
  Row now = row_at(i0);
  bool ok = true;
  for (uint32_t phase = 0; ok && i0 < total; i0 += stride, phase ^= 1) {
    const bool there = now.from >= 0;
    const int rows = __popc(__ballot_sync(0xffffffffu, there));
    if (lane == 0) bar_expect_tx(&sh.bar[warp], uint32_t(rows * a.row_bytes));
    __syncwarp();
    if (there) bulk_g2s(buf + lane * a.row_bytes, base + now.from, uint32_t(a.row_bytes), &sh.bar[warp]);
    const Row next = row_at(i0 + stride);
    if (there) {
      if (lane & 1)
        a.place[now.d] = __ldcg(a.place + now.s);
      else
        a.weight[now.d] = __ldcg(a.weight + now.s);
    }
    ok = __all_sync(0xffffffffu, bar_wait(&sh.bar[warp], phase, a.err));
    if (!ok) bar_wait(&sh.bar[warp], phase, a.err, kSpinCyclesAfterError);  // the copies in flight land before the CTA leaves
    if (ok && there)
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(base + now.to), "r"(sa(buf + lane * a.row_bytes)),
                   "r"(uint32_t(a.row_bytes))
                   : "memory");
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();  // every lane's row has been read: the buffer may be filled again
    now = next;
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  static OnEveryDevice ready;
  const cudaError_t e =
      ready([] { return cudaFuncSetAttribute(cache_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kEvSmem)); });
  if (e != cudaSuccess) return e;
  const int64_t units = int64_t(a.n_req) * a.hkv, most = a.width << a.page_shift;
  // As many CTAs a unit as the SMs hold, where several of more than 256 places of the table each (a request may fill fewer).  80 heads of up to 8003 keys to 2048, us: 1 CTA each 80, 2 62, 4
  // (a few of them left over for a second turn) 60, 8 75.
  unsigned C = 1;
  while (C < unsigned(kEvMost) && units * C * 2 <= 3 * sm_count() && most > int64_t(C) * 512) C *= 2;
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
