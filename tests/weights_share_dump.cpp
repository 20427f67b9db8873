// Runs the share arithmetic of the gathered attention weights (gsi_weights_share.cuh)
// on the CPU and prints what every CTA would take, for test_weights_share_cpu.py.
// The threads of a block are fibers of one host thread, which change over at the
// warps' exchanges and the block's barriers.
//
// Input, a case a line: KT GRID TPT HKV CAUSAL PAGE_SHIFT WIDTH N N_REQ
// q_start[0 .. N_REQ] kv_len[0 .. N_REQ - 1] held[0 .. N_REQ - 1]
// Output, a line a case: {"total": ..., "alike": every thread found the same share,
// "ctas": [[[r, h, t, u0, n, a, b, b0, b1], ...], ...]}
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

constexpr int kMaxThreads = 448;
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
static unsigned __ballot_sync(unsigned, bool p) {
  const long long* all = warp_meet(p);
  unsigned bits = 0;
  for (int i = 0; i < 32; ++i) bits |= unsigned(all[i]) << i;
  return bits;
}
static int __popc(unsigned x) { return __builtin_popcount(x); }
static void __syncthreads() { g_block.meet(threadIdx.x, 0); }
static int __ffs(int x) { return __builtin_ffs(x); }

#include "gsi_weights_share.cuh"

static gsi::KeyWeightArgs g_args;
static int g_tpt;
template <int KT>
struct Walks {
  static gsi::KwWalk<KT> of[kMaxThreads];
};
template <int KT>
gsi::KwWalk<KT> Walks<KT>::of[kMaxThreads];

template <int KT, int NT>
static void body() {
  gsi::KwWalk<KT> w;
  gsi::kw_share<KT, NT>(g_args, g_tpt, w);
  Walks<KT>::of[threadIdx.x] = w;
  g_done[threadIdx.x] = true;
  for (;;) swapcontext(&g_fiber[threadIdx.x], &g_main);
}

template <int KT, int NT>
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
    makecontext(&g_fiber[t], body<KT, NT>, 0);
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

template <int KT, int NT>
static void run(const gsi::KeyWeightArgs& a, int grid) {
  bool alike = true;
  for (int c = 0; c < grid; ++c) {
    blockIdx.x = c;
    run_block<KT, NT>();
    auto* all = Walks<KT>::of;
    for (int t = 1; t < NT; ++t) {
      alike &= all[0].pos == all[t].pos && all[0].end == all[t].end;
      if (all[0].pos < all[0].end)
        alike &= all[0].total == all[t].total && all[0].grid == all[t].grid && all[0].r == all[t].r && all[0].h == all[t].h &&
                 all[0].t == all[t].t && all[0].off == all[t].off;
    }
    gsi::KwWalk<KT> w = all[0];
    std::printf("%s[", c ? ", " : "{\"ctas\": [");
    gsi::KwSeg g;
    for (int i = 0; w.next(a, g); ++i) {
      int b0 = 0, b1 = 0;
      w.parts(g, b0, b1);
      std::printf("%s[%d, %d, %d, %d, %d, %d, %d, %d, %d]", i ? ", " : "", g.r, g.h, g.t, g.u0, g.n, g.a, g.b, b0, b1);
    }
    std::printf("]");
  }
  std::printf("], \"alike\": %d}\n", int(alike));
}

static long long number() {
  long long v = 0;
  if (std::scanf("%lld", &v) != 1) return -1;
  return v;
}

int main() {
  int kt;
  while (std::scanf("%d", &kt) == 1) {
    const int grid = int(number());
    g_tpt = int(number());
    gsi::KeyWeightArgs& a = g_args = gsi::KeyWeightArgs{};
    a.hkv = int(number());
    a.causal = int(number());
    a.page_shift = int(number());
    a.width = number();
    a.N = int(number());
    a.n_req = int(number());
    std::vector<int32_t> start(a.n_req + 1), len(a.n_req + 1), held(a.n_req + 1);
    for (int i = 0; i <= a.n_req; ++i) start[i] = int(number());
    for (int i = 0; i < a.n_req; ++i) len[i] = int(number());
    for (int i = 0; i < a.n_req; ++i) held[i] = int(number());
    a.q_start = start.data();
    a.kv_len = len.data();
    a.held = held.data();
    gridDim.x = grid;
    if (kt == 64) run<64, 256>(a, grid); else if (kt == 128) run<128, 448>(a, grid); else run<256, 448>(a, grid);
  }
  return 0;
}
