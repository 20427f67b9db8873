// Runs the attention kernels' share arithmetic (gsi_attn_share.cuh) on the CPU
// and prints what every CTA would take, for test_attn_share_cpu.py.  The threads
// of a block are fibers of one host thread, which change over at the warps'
// exchanges and the block's barriers.
//
// Input, a case a line: NT GRID UT KT EXTRA HKV GROUP CAUSAL WINDOW PAGE_SHIFT WIDTH N N_REQ
// q_start[0 .. N_REQ] kv_len[0 .. N_REQ - 1]
// Output, a line a case: {"grid": ..., "total": ..., "dealt": ..., "alike": every thread found the same share,
// "ctas": [[[r, h, u, t0, n, a, b, b0, b1], ...], ...]}
#include <cuda_runtime.h>
#include <ucontext.h>

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <vector>

#undef __device__
#undef __forceinline__
#undef __noinline__
#undef __shared__
#undef __host__
#define __device__
#define __host__
#define __forceinline__ inline
#define __noinline__ __attribute__((noinline))
#define __shared__ static

using std::max;
using std::min;

struct Index {
  unsigned x;
};
static Index threadIdx, blockIdx, gridDim;

constexpr int kMaxThreads = 384;
static ucontext_t g_main, g_fiber[kMaxThreads];
static bool g_done[kMaxThreads];
static std::vector<char> g_stacks(size_t(kMaxThreads) * 65536);

// A warp or a block: values of its threads, once all are there.
struct Group;
static Group* g_waits[kMaxThreads];  // for whom a thread waits
static unsigned g_since[kMaxThreads];
struct Group {
  int n = 0, arrived = 0;
  unsigned generation = 0;
  long long in[kMaxThreads], out[kMaxThreads];
  const long long* meet(int i, long long v) {
    const unsigned mine = generation;
    in[i] = v;
    if (++arrived == n) {
      std::memcpy(out, in, sizeof(long long) * n);
      arrived = 0;
      ++generation;
    } else {
      g_waits[threadIdx.x] = this;
      g_since[threadIdx.x] = mine;
      swapcontext(&g_fiber[threadIdx.x], &g_main);
    }
    return out;
  }
};
static Group g_block, g_warp[kMaxThreads / 32];

static const long long* warp_meet(long long v) { return g_warp[threadIdx.x / 32].meet(threadIdx.x % 32, v); }
template <class T>
static T __ldcg(const T* p) {
  return *p;
}
template <class T>
static T __shfl_up_sync(unsigned, T v, int o) {
  const long long* all = warp_meet(v);
  const int lane = threadIdx.x % 32;
  return lane >= o ? T(all[lane - o]) : v;
}
template <class T>
static T __shfl_sync(unsigned, T v, int from) {
  return T(warp_meet(v)[from]);
}
static unsigned __ballot_sync(unsigned, bool p) {
  const long long* all = warp_meet(p);
  unsigned bits = 0;
  for (int i = 0; i < 32; ++i) bits |= unsigned(all[i]) << i;
  return bits;
}
static void __syncthreads() { g_block.meet(threadIdx.x, 0); }
static int __syncthreads_or(int p) {
  const long long* all = g_block.meet(threadIdx.x, p != 0);
  return std::any_of(all, all + g_block.n, [](long long x) { return x != 0; });
}
static int __popc(unsigned x) { return __builtin_popcount(x); }
static int __ffs(int x) { return __builtin_ffs(x); }

#include "gsi_attn_share.cuh"

static gsi::AttnArgs g_args;
static int g_ut, g_kt, g_extra;
static gsi::AttnWalk g_walk[kMaxThreads];

template <int NT>
static void body() {
  gsi::AttnWalk w;
  w.ut = g_ut;
  w.kt = g_kt;
  w.s = gsi::attn_share<NT>(g_args, g_ut, g_kt, g_extra, w.p);
  g_walk[threadIdx.x] = w;
  g_done[threadIdx.x] = true;
  for (;;) swapcontext(&g_fiber[threadIdx.x], &g_main);
}

template <int NT>
static void run_block() {
  g_block.n = NT;
  for (int t = 0; t < NT; ++t) {
    g_warp[t / 32].n = 32;
    g_done[t] = false;
    g_waits[t] = nullptr;
    getcontext(&g_fiber[t]);
    g_fiber[t].uc_stack.ss_sp = &g_stacks[size_t(t) * 65536];
    g_fiber[t].uc_stack.ss_size = 65536;
    g_fiber[t].uc_link = nullptr;
    makecontext(&g_fiber[t], body<NT>, 0);
  }
  for (bool more = true; more;) {
    more = false;
    for (int t = 0; t < NT; ++t)
      if (!g_done[t]) {
        more = true;
        if (g_waits[t] && g_waits[t]->generation == g_since[t]) continue;
        g_waits[t] = nullptr;
        threadIdx.x = t;
        swapcontext(&g_main, &g_fiber[t]);
      }
  }
}

static long long number() {
  long long v = 0;
  if (std::scanf("%lld", &v) != 1) return -1;
  return v;
}

int main() {
  int nt;
  while (std::scanf("%d", &nt) == 1) {
    const int grid = int(number());
    g_ut = int(number());
    g_kt = int(number());
    g_extra = int(number());
    gsi::AttnArgs& a = g_args = gsi::AttnArgs{};
    a.hkv = int(number());
    a.group = int(number());
    a.causal = int(number());
    a.window = int(number());
    a.page_shift = int(number());
    a.width = number();
    a.N = int(number());
    a.n_req = int(number());
    std::vector<int32_t> start(a.n_req + 1), len(a.n_req + 1);
    for (int i = 0; i <= a.n_req; ++i) start[i] = int(number());
    for (int i = 0; i < a.n_req; ++i) len[i] = int(number());
    a.q_start = start.data();
    a.kv_len = len.data();
    gridDim.x = grid;
    bool alike = true;
    for (int c = 0; c < grid; ++c) {
      blockIdx.x = c;
      if (nt == 384) run_block<384>(); else run_block<256>();
      for (int t = 1; t < nt; ++t) {
        const gsi::AttnWalk &x = g_walk[0], &y = g_walk[t];
        alike &= x.s.total == y.s.total && x.s.pos == y.s.pos && x.s.end == y.s.end && x.s.grid == y.s.grid &&
                 x.s.extra == y.s.extra && x.s.dealt == y.s.dealt;
        if (x.s.pos < x.s.end || x.s.dealt > 0)
          alike &= x.p.r == y.p.r && x.p.h == y.p.h && x.p.u == y.p.u && x.p.off == y.p.off && x.p.q.q0 == y.p.q.q0 &&
                   x.p.q.q_len == y.p.q.q_len && x.p.q.len == y.p.q.len;
      }
      gsi::AttnWalk w = g_walk[0];
      if (c == 0)
        std::printf("{\"grid\": %d, \"total\": %lld, \"extra\": %d, \"dealt\": %d, \"ctas\": [", w.s.grid, w.s.total, w.s.extra,
                    w.s.dealt);
      std::printf("%s[", c ? ", " : "");
      gsi::AttnSeg g;
      for (int i = 0; w.next(a, g); ++i) {
        int b0 = 0, b1 = 0;
        if (w.s.dealt == 0) w.parts(g, b0, b1);
        std::printf("%s[%d, %d, %d, %d, %d, %d, %d, %d, %d]", i ? ", " : "", g.r, g.h, g.u, g.t0, g.n, g.a, g.b, b0, b1);
      }
      std::printf("]");
    }
    std::printf("], \"alike\": %d}\n", int(alike));
  }
  return 0;
}
