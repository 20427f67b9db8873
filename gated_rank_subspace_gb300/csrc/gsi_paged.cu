// Pages of the key/value cache: the plan of a step's pages and slots, the
// return of pages, and the append of a qkv map's rows at their slots.

#include "gsi_append.cuh"
#include "gsi_kernels.h"

namespace gsi {

// ------------------------------------------------------------------ plan
// For request r with c_r cached and f_r fresh tokens and pages of P tokens:
//   S_r = sum_{i<r} f_i          (q_start)
//   n_r = ceil((c_r + f_r) / P) - ceil(c_r / P),   A_r = sum_{i<r} n_i
// page j >= ceil(c_r / P) of r is free[n_free - 1 - (A_r + j - ceil(c_r / P))],
// and token t of r, at place p = c_r + t - S_r, has the slot
// page(r, p / P) * P + p % P.
//
// Bound: latency at a server's sizes (16 B a token are written): 3.8 us for 16
// requests, 9.4 us for 4093 with 74,000 tokens (a launch alone is ~2).  Every CTA
// forms both prefix sums itself -- a second launch or a grid barrier costs
// more than reading 8 B a request again from L2 -- and writes its own slice
// of the tokens, each finding its request by bisection of the prefix in
// shared memory.  A new page begins with a new token, so the CTA that writes
// that token also writes the table entry, and no CTA reads an entry that
// another one writes.
constexpr int kPlanThreads = 512;
constexpr int kPlanItems = 8;                          // requests a thread takes of a chunk
constexpr int kPlanChunk = kPlanThreads * kPlanItems;  // requests whose prefix sums are in shared memory
constexpr int kPlanTokens = 512;                       // new tokens of a CTA, at least
constexpr int kPlanSmem = (3 * kPlanChunk + 1) * 4;

struct PlanSums {
  long long fresh, pages;
  unsigned bad;  // GSI_PLAN_ bits, or-ed
};

// What a request adds, or why it cannot be planned.
__device__ __forceinline__ PlanSums plan_request(const PlanArgs& a, int cached, int fresh) {
  const int shift = a.page_shift;
  const long long round = (1ll << shift) - 1, end = (long long)cached + fresh;
  if (cached < 0 || fresh < 0 || end > 0x7fffffffll) return PlanSums{0, 0, GSI_PLAN_BAD_LENGTH};
  const long long held = (cached + round) >> shift, want = (end + round) >> shift;
  return PlanSums{fresh, want - held, want > a.width ? unsigned(GSI_PLAN_TABLE_FULL) : 0u};
}

// Exclusive prefix over the block's threads; *total is the block's sum.
__device__ __forceinline__ PlanSums plan_scan(PlanSums v, PlanSums* warp_sums, PlanSums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  PlanSums inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long f = __shfl_up_sync(0xffffffffu, inc.fresh, o), p = __shfl_up_sync(0xffffffffu, inc.pages, o);
    if (lane >= o) inc.fresh += f, inc.pages += p;
  }
  inc.bad = __reduce_or_sync(0xffffffffu, v.bad);
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  PlanSums before{0, 0, 0}, all{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const PlanSums s = warp_sums[w];
    if (w < warp) before.fresh += s.fresh, before.pages += s.pages;
    all.fresh += s.fresh, all.pages += s.pages, all.bad |= s.bad;
  }
  *total = all;
  return PlanSums{before.fresh + inc.fresh - v.fresh, before.pages + inc.pages - v.pages, 0};
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int plan_smem[];
  __shared__ PlanSums s_warp[kPlanThreads / 32];
  int* s_start = plan_smem;                // S_r of the chunk's requests, and their end
  int* s_pages = s_start + kPlanChunk + 1;  // A_r
  int* s_cached = s_pages + kPlanChunk;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, shift = a.page_shift;
  const int round = (1 << shift) - 1;
  const int n_free = __ldcg(a.n_free);
  const bool one_chunk = a.n_req <= kPlanChunk;

  int c[kPlanItems], f[kPlanItems];
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const int r = c0 + tid * kPlanItems + i;
      c[i] = f[i] = 0;
      if (r < a.n_req) {
        c[i] = __ldcg(a.cached + r);
        f[i] = __ldcg(a.fresh + r);
      }
    }
  };
  auto sums = [&]() {
    PlanSums s{0, 0, 0};
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const PlanSums q = plan_request(a, c[i], f[i]);
      s.fresh += q.fresh, s.pages += q.pages, s.bad |= q.bad;
    }
    return s;
  };

  // 1. totals and checks, before anything is written
  PlanSums all, at;
  if (one_chunk) {
    load(0);
    at = plan_scan(sums(), s_warp, &all);
  } else {
    PlanSums mine{0, 0, 0};
    for (int r = tid; r < a.n_req; r += kPlanThreads) {
      const PlanSums q = plan_request(a, __ldcg(a.cached + r), __ldcg(a.fresh + r));
      mine.fresh += q.fresh, mine.pages += q.pages, mine.bad |= q.bad;
    }
    plan_scan(mine, s_warp, &all);
  }
  unsigned bad = all.bad;
  if (n_free < 0 || n_free > a.capacity || all.pages > n_free) bad |= GSI_PLAN_NO_PAGES;
  if (all.fresh > a.n_tokens) bad |= GSI_PLAN_TOO_MANY_TOKENS;

  const int n_new = bad ? 0 : int(all.fresh);
  // this CTA's tokens
  const int t0 = int((long long)a.n_tokens * blockIdx.x / gridDim.x);
  const int t1 = int((long long)a.n_tokens * (blockIdx.x + 1) / gridDim.x);
  for (int t = max(t0, n_new) + tid; t < t1; t += kPlanThreads) {
    a.slots[t] = -1;
    a.token_req[t] = -1;
    a.positions[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    *a.status = int(bad);
    *a.n_free_out = bad ? n_free : int(n_free - all.pages);
    a.q_start[a.n_req] = n_new;
  }
  if (bad) {
    if (blockIdx.x == 0)
      for (int r = tid; r < a.n_req; r += kPlanThreads) {
        a.q_start[r] = 0;
        a.kv_len[r] = max(0, __ldcg(a.cached + r));
      }
    return;
  }

  // 2. the requests, a chunk at a time
  PlanSums base{0, 0, 0};
  for (int c0 = 0; c0 < a.n_req; c0 += kPlanChunk) {
    const int n = min(kPlanChunk, a.n_req - c0);
    PlanSums chunk = all;
    if (!one_chunk) {
      load(c0);
      at = plan_scan(sums(), s_warp, &chunk);
    }
    int s = int(base.fresh + at.fresh), q = int(base.pages + at.pages);
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const int r = tid * kPlanItems + i;
      if (r < n) {
        s_start[r] = s;
        s_pages[r] = q;
        s_cached[r] = c[i];
        if (blockIdx.x == 0) {
          a.q_start[c0 + r] = s;
          a.kv_len[c0 + r] = c[i] + f[i];
        }
      }
      s += f[i];
      q += ((c[i] + f[i] + round) >> shift) - ((c[i] + round) >> shift);
    }
    const int first = int(base.fresh), end = int(base.fresh + chunk.fresh);
    if (tid == 0) s_start[n] = end;
    __syncthreads();
    for (int t = max(t0, first) + tid; t < min(t1, end); t += kPlanThreads) {
      int lo = 0, hi = n;  // the last request that begins at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= t) lo = mid; else hi = mid;
      }
      const int64_t r = c0 + lo;
      const int cached = s_cached[lo], pos = cached + t - s_start[lo];
      const int held = (cached + round) >> shift, j = pos >> shift;
      int id;
      if (j >= held) {
        id = __ldcg(a.free_pages + (n_free - 1 - (s_pages[lo] + j - held)));
        if ((pos & round) == 0) a.table[r * a.width + j] = id;
      } else {
        id = __ldcg(a.table + r * a.width + j);
      }
      a.slots[t] = id < 0 ? -1 : ((long long)id << shift) + (pos & round);
      a.token_req[t] = int(r);
      a.positions[t] = pos;
    }
    base.fresh += chunk.fresh;
    base.pages += chunk.pages;
    __syncthreads();  // before the next chunk's prefix sums overwrite these
  }
}

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s) {
  static OnEveryDevice ready;
  const cudaError_t e =
      ready([] { return cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmem); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(max(1, min(sm_count(), a.n_tokens / kPlanTokens)));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = kPlanSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
}

// ------------------------------------------------------------------ trim
// Request r filled ceil(l_r / P) pages and now fills ceil(k_r / P): the pages
// between go back on the stack, F_r of them behind the B_r = sum_{i<r} F_i of
// the requests before.  The i-th page given back (in the order of requests and
// pages) lands at n_free + F - 1 - i, so a plan that needs them again takes
// them in the same order.  As in the plan, every CTA forms the prefix sums
// itself and writes its own slice of the pages, each finding its request by
// bisection.  Latency bounds it: 2.9 us for 16 requests, 5.2 for 4093.
constexpr int kTrimPages = 1024;  // places of the stack a CTA, at least (what is given back may be less)

__device__ __forceinline__ PlanSums trim_request(const TrimArgs& a, int len, int kept) {
  const long long round = (1ll << a.page_shift) - 1;
  if (len < 0 || kept < 0 || kept > len) return PlanSums{0, 0, GSI_PLAN_BAD_LENGTH};
  const long long held = (len + round) >> a.page_shift;
  return PlanSums{0, held - ((kept + round) >> a.page_shift), held > a.width ? unsigned(GSI_PLAN_TABLE_FULL) : 0u};
}

__global__ void __launch_bounds__(kPlanThreads) paged_trim_kernel(const __grid_constant__ TrimArgs a) {
  __shared__ PlanSums s_warp[kPlanThreads / 32];
  __shared__ int s_back[kPlanChunk], s_first[kPlanChunk];  // B_r, and the first page that r gives back
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, shift = a.page_shift, round = (1 << shift) - 1;
  const int n_free = __ldcg(a.n_free);
  const bool one_chunk = a.n_req <= kPlanChunk;
  int len[kPlanItems], kept[kPlanItems];
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const int r = c0 + tid * kPlanItems + i;
      len[i] = kept[i] = 0;
      if (r < a.n_req) {
        len[i] = __ldcg(a.kv_len + r);
        kept[i] = __ldcg(a.kept + r);
      }
    }
  };
  auto sums = [&]() {
    PlanSums s{0, 0, 0};
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const PlanSums q = trim_request(a, len[i], kept[i]);
      s.pages += q.pages, s.bad |= q.bad;
    }
    return s;
  };

  // 1. the total and the checks, before anything is written
  PlanSums all, at;
  if (one_chunk) {
    load(0);
    at = plan_scan(sums(), s_warp, &all);
  } else {
    PlanSums mine{0, 0, 0};
    for (int r = tid; r < a.n_req; r += kPlanThreads) {
      const PlanSums q = trim_request(a, __ldcg(a.kv_len + r), __ldcg(a.kept + r));
      mine.pages += q.pages, mine.bad |= q.bad;
    }
    plan_scan(mine, s_warp, &all);
  }
  unsigned bad = all.bad;
  if (n_free < 0 || n_free > a.capacity || n_free + all.pages > a.capacity) bad |= GSI_PLAN_NO_PAGES;
  if (blockIdx.x == 0 && tid == 0) {
    *a.status = int(bad);
    *a.n_free_out = bad ? n_free : int(n_free + all.pages);
  }
  if (bad) return;

  // 2. the requests, a chunk at a time
  const int total = int(all.pages);
  const int i0 = int(all.pages * blockIdx.x / gridDim.x), i1 = int(all.pages * (blockIdx.x + 1) / gridDim.x);
  int base = 0;
  for (int c0 = 0; c0 < a.n_req; c0 += kPlanChunk) {
    const int n = min(kPlanChunk, a.n_req - c0);
    PlanSums chunk = all;
    if (!one_chunk) {
      load(c0);
      at = plan_scan(sums(), s_warp, &chunk);
    }
    int b = base + int(at.pages);
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
      const int r = tid * kPlanItems + i, first = int(((long long)kept[i] + round) >> shift);
      if (r < n) {
        s_back[r] = b;
        s_first[r] = first;
      }
      b += int(((long long)len[i] + round) >> shift) - first;
    }
    __syncthreads();
    const int end = base + int(chunk.pages);
    for (int i = max(i0, base) + tid; i < min(i1, end); i += kPlanThreads) {
      int lo = 0, hi = n;  // the last request whose pages begin at or before i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_back[mid] <= i) lo = mid; else hi = mid;
      }
      a.free_pages[n_free + total - 1 - i] = __ldcg(a.table + int64_t(c0 + lo) * a.width + s_first[lo] + i - s_back[lo]);
    }
    base = end;
    __syncthreads();  // before the next chunk's sums overwrite these
  }
}

cudaError_t launch_paged_trim(const TrimArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  // (the pages given back are at most the stack's places)
  cfg.gridDim = dim3(unsigned(max(int64_t(1), min(int64_t(sm_count()), a.capacity / kTrimPages))));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_trim_kernel, a);
}

// ------------------------------------------------------------------ append
// A copy: (hq + 2 hkv) * dim values a token are read, converted and written
// once, so the bytes bound it (2048 tokens of 16 + 2 x 16 heads of 256: 24 us,
// 6.3 TB/s; 16 tokens 1.9 us).  A CTA takes up to 512 16-byte output vectors of
// one token; its slot is one broadcast load.
constexpr int kAppendThreads = 256;

template <class XT, class CT>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(AppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int64_t slot = __ldcg(reinterpret_cast<const long long*>(a.slots) + t);
  const bool there = slot >= 0 && slot < a.n_slots;
  const int64_t pg = slot >> a.page_shift, off = slot & ((int64_t(1) << a.page_shift) - 1);
  const int per_head = a.dim / CT::kPerVec;
  const int n_vec = (a.hq + 2 * a.hkv) * per_head;
  const char* row = static_cast<const char*>(a.X) + t * a.row_stride * XT::kBytes;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int v = (blockIdx.y * 2 + i) * kAppendThreads + threadIdx.x;
    if (v >= n_vec) return;
    int head = v / per_head;
    const int e = (v - head * per_head) * CT::kPerVec;
    char* dst;
    if (head < a.hq) {
      if (!a.Q) continue;
      dst = static_cast<char*>(a.Q) + ((t * a.hq + head) * a.dim + e) * CT::kBytes;
    } else {
      if (!there) return;
      head -= a.hq;
      const bool val = head >= a.hkv;
      if (val) head -= a.hkv;
      dst = static_cast<char*>(val ? a.V : a.K) +
            (pg * a.page_stride + head * a.head_stride + off * a.token_stride + e) * CT::kBytes;
    }
    *reinterpret_cast<uint4*>(dst) = append_vec<XT, CT>(row, int64_t(v) * CT::kPerVec);
  }
}

cudaError_t launch_cache_append(const AppendArgs& a, gsi_dtype xdt, gsi_dtype cdt, cudaStream_t s) {
  const int n_vec = (a.hq + 2 * a.hkv) * (a.dim / (cdt == GSI_BF16 ? 8 : 4));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.T, (n_vec + 2 * kAppendThreads - 1) / (2 * kAppendThreads));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (xdt == GSI_F32)
    return cdt == GSI_F32 ? cudaLaunchKernelEx(&cfg, cache_append_kernel<F32, F32>, a)
                          : cudaLaunchKernelEx(&cfg, cache_append_kernel<F32, BF16>, a);
  return cdt == GSI_F32 ? cudaLaunchKernelEx(&cfg, cache_append_kernel<BF16, F32>, a)
                        : cudaLaunchKernelEx(&cfg, cache_append_kernel<BF16, BF16>, a);
}

}  // namespace gsi
