// Verification of drafted tokens against the target's probabilities.

#include "gsi_common.cuh"
#include "gsi_kernels.h"

namespace gsi {

// A request's rows q_start[r] .. q_start[r + 1) hold its last token and its n
// drafts; row t's probabilities p (target) and q (draft) are those of the token
// behind it.  Draft d of row t stands if u_t q(d) < p(d); the first that does not
// is replaced by a token of the distribution max(p - q, 0), and behind n standing
// drafts comes one of p:  the smallest token x with
//   sum_{y <= x} m(y) > v sum_y m(y).
// Sums of 10^5 probabilities have to be right to far below one of them, whatever
// their order: p and q become whole multiples of 2^-46 (exact from 2^-23 on), whose
// differences and sums are exact: in 64 bits below 2^18 tokens (rows need not add
// up to 1, and 2^18 tokens of 1 are 2^64); from there on a lane's sum has 64 bits (2^24
// tokens are 2^16 a lane of one CTA, 2^62), those of warps, CTAs and the row
// 128.  (128 bits for all: one row of 50257 7.8 us instead of 7.3, 16 of 250002 15.3
// instead of 14.2.)
//
// A cluster takes a request.  Every CTA finds the row (the drafts' probabilities
// are a few loads), then each sums a stretch of the row, a warp a stretch of that;
// the CTA whose stretch holds the token looks through the warp's part of it again,
// all its threads four tokens each.  The bytes of the one row of p and q bound it,
// for few requests the chain of loads and exchanges (one row of 50257 7 us, 64 of
// 100003 20, 16 of 250002 bf16 probabilities 18, which take 25 one value at a time).
constexpr int kVfThreads = 256, kVfWarps = kVfThreads / 32, kVfMost = 8;
constexpr int kVfUnroll = 2;  // groups of 8 tokens of each row in flight a lane

// A probability within 0 .. 1 (NaN: 0) as hi 2^-23 + lo 2^-46, both rounded to nearest: adding 1 leaves x's multiple of
// 2^-23 in the sum's lower bits, and the rest, which is exact, added to 1.5 2^-23 its multiple of 2^-46.  (Conversions to
// 64-bit numbers run at a fraction of the rate: 88 us with them where this takes 20, 64 rows of 100003.)
__device__ __forceinline__ int2 vf_split(float x) {
  x = __saturatef(x);
  const float h = __fadd_rn(x, 1.f), l = __fadd_rn(__fsub_rn(x, __fsub_rn(h, 1.f)), 0x1.8p-23f);
  return make_int2(__float_as_int(h) - __float_as_int(1.f), __float_as_int(l) - __float_as_int(0x1.8p-23f));
}

// Eight values from element e on (a multiple of 16 bytes), or zeros.
template <class T>
__device__ __forceinline__ void vf_load8(const void* base, int64_t e, bool there, float (&f)[8]) {
  const char* at = static_cast<const char*>(base) + e * T::kBytes;
#pragma unroll
  for (int i = 0; i < 8; i += T::kPerVec) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (there) v = ld_cg_v4(at + i * T::kBytes);
    T::unpack(v, f + i);
  }
}

constexpr int kVfWide = 1 << 18;  // tokens from which on a row's sum may pass 64 bits

template <class Sum>
struct VfShared {
  Sum total;  // of this CTA (read by the cluster)
  Sum warps[kVfWarps];
  int fail;
};

// A lane's sum over its warp.
template <class Sum>
__device__ __forceinline__ Sum vf_warp_sum(unsigned long long sum) {
  unsigned long long low = sizeof(Sum) > 8 ? sum & 0xffffffffu : sum, high = sum >> 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    low += __shfl_xor_sync(0xffffffffu, low, o);
    if constexpr (sizeof(Sum) > 8) high += __shfl_xor_sync(0xffffffffu, high, o);
  }
  if constexpr (sizeof(Sum) > 8) return (Sum(high) << 32) + low;
  return low;
}
// floor(total v 2^-64)
template <class Sum>
__device__ __forceinline__ Sum vf_share(Sum total, unsigned long long v) {
  const Sum low = __umul64hi((unsigned long long)total, v);
  if constexpr (sizeof(Sum) > 8) return Sum((unsigned long long)(total >> 64)) * v + low;
  return low;
}

template <class TT, class DT, class Sum>
__global__ void __launch_bounds__(kVfThreads, 4) verify_drafts_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ VfShared<Sum> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), c = int(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / C;
  pdl_launch_dependents();
  if (tid == 0) sh.fail = 0x7fffffff;
  pdl_wait();
  const int t0 = min(max(__ldcg(a.q_start + r), 0), a.N), t1 = min(max(__ldcg(a.q_start + r + 1), t0), a.N);
  const int n = t1 - t0 - 1;  // drafts
  if (n < 0) {
    if (c == 0 && tid == 0) {
      a.accepted[r] = 0;
      if (a.kept) a.kept[r] = __ldcg(a.kv_len + r);
    }
    return;  // the whole cluster
  }
  __syncthreads();

  // ---- the first draft that does not stand, by what its probabilities count as (NaN and what is negative 0, above 1 as 1)
  auto p_at = [&](int t, int x) { return TT::load1_cg(a.target, t * a.target_stride + x); };
  auto q_at = [&](int t, int x) { return a.draft ? DT::load1_cg(a.draft, t * a.draft_stride + x) : 1.f; };
  for (int i = tid; i < n; i += kVfThreads) {
    const int t = t0 + i, d = __ldcg(a.tokens + t + 1);
    // (the product of two float32 is exact in 64 bits; a token outside the vocabulary has no probability)
    const bool stands = d >= 0 && d < a.vocab && double(__ldcg(a.uniforms + t)) * double(__saturatef(q_at(t, d))) < double(__saturatef(p_at(t, d)));
    if (!stands) {
      atomicMin(&sh.fail, i);
      break;
    }
  }
  __syncthreads();
  const int taken = min(sh.fail, n);
  const int t = t0 + taken;
  const int gone = taken < n && !a.draft ? __ldcg(a.tokens + t + 1) : -1;  // a certain draft's whole mass

  // ---- the distribution, a stretch a CTA and a warp
  const int x0 = int(int64_t(a.vocab) * c / C), x1 = int(int64_t(a.vocab) * (c + 1) / C);
  const int y0 = x0 + int(int64_t(x1 - x0) * warp / kVfWarps), y1 = x0 + int(int64_t(x1 - x0) * (warp + 1) / kVfWarps);
  bool left = taken < n;  // what the draft leaves of the target, else the target itself
  // the mass of a token with probabilities p and q, in units of 2^-46
  auto mass = [&](float p, float q, int x) -> long long {
    const int2 u = vf_split(p);
    if (!left) return (long long)u.x * (1 << 23) + u.y;
    if (!a.draft) return x == gone ? 0 : (long long)u.x * (1 << 23) + u.y;
    const int2 w = vf_split(q);
    // (the split is monotone; NaN compares as 0)
    const long long m = (long long)(u.x - w.x) * (1 << 23) + (u.y - w.y);
    return m > 0 ? m : 0;
  };
  const bool both = a.draft != nullptr;
  for (;;) {
    unsigned long long sum = 0;
    // 16 bytes at a time where the rows' addresses allow it (an odd vocabulary's do from some token on, both rows alike where
    // their types are), one by one before and behind
    const bool two = both && left;
    const int64_t pr = t * a.target_stride, qr = two ? t * a.draft_stride : 0;
    auto one = [&](int x) { sum += mass(TT::load1_cg(a.target, pr + x), two ? DT::load1_cg(a.draft, qr + x) : 0.f, x); };
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.target) + (pr + y0) * TT::kBytes;
    int z0 = y0 + int((16 - (pa & 15)) & 15) / TT::kBytes, z1 = z0;
    if (z0 < y1 && (!two || ((reinterpret_cast<uintptr_t>(a.draft) + (qr + z0) * DT::kBytes) & 15) == 0)) z1 = z0 + (y1 - z0) / 8 * 8;
    z0 = min(z0, z1 = min(z1, y1));
    for (int x = y0 + lane; x < z0; x += 32) one(x);
    for (int x = z0 + 8 * lane; x < z1; x += 256 * kVfUnroll) {
      float p[kVfUnroll][8], q[kVfUnroll][8];
#pragma unroll
      for (int i = 0; i < kVfUnroll; ++i) vf_load8<TT>(a.target, pr + x + 256 * i, x + 256 * i < z1, p[i]);
#pragma unroll
      for (int i = 0; i < kVfUnroll; ++i) vf_load8<DT>(a.draft, qr + x + 256 * i, two && x + 256 * i < z1, q[i]);
#pragma unroll
      for (int i = 0; i < kVfUnroll; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += mass(p[i][e], q[i][e], x + 256 * i + e);
    }
    for (int x = z1 + lane; x < y1; x += 32 * 8) {
      float p[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = x + 32 * i < y1 ? TT::load1_cg(a.target, pr + x + 32 * i) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = two && x + 32 * i < y1 ? DT::load1_cg(a.draft, qr + x + 32 * i) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += mass(p[i], q[i], x + 32 * i);
    }
    const Sum mine = vf_warp_sum<Sum>(sum);
    if (lane == 0) sh.warps[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      Sum s = 0;
      for (int w = 0; w < kVfWarps; ++w) s += sh.warps[w];
      sh.total = s;
    }
    cluster.sync();
    Sum total = 0, base = 0;
    for (int b = 0; b < C; ++b) {
      if (b == c) base = total;
      total += *cluster.map_shared_rank(&sh.total, b);
    }
    cluster.sync();  // the totals have been read
    if (total == 0) {
      if (left) {  // a draft that leaves nothing: the target itself
        left = false;
        continue;
      }
      if (c == 0 && tid == 0) a.out[t] = -1;  // a row without any mass
      break;
    }
    // the token's mass ends above floor(v total)
    const float v = fminf(fmaxf(__ldcg(a.samples + r), 0.f), 0x1.fffffep-1f);
    const Sum at = vf_share(total, __float2ull_rz(v * 18446744073709551616.f));
    if (at < base || at >= base + sh.total) break;  // in another CTA's stretch
    int w = 0;
    for (; at >= base + sh.warps[w]; ++w) base += sh.warps[w];
    const int f0 = x0 + int(int64_t(x1 - x0) * w / kVfWarps), f1 = x0 + int(int64_t(x1 - x0) * (w + 1) / kVfWarps);
    for (int z = f0; z < f1; z += 4 * kVfThreads) {
      long long m[4];
      float p[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = z + 4 * tid + i;
        p[i] = x < f1 ? p_at(t, x) : 0.f;
        q[i] = both && left && x < f1 ? q_at(t, x) : 0.f;
      }
      unsigned long long mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) mine += m[i] = mass(p[i], q[i], z + 4 * tid + i);
      unsigned long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncthreads();  // the sums before have been read
      if (lane == 31) sh.warps[warp] = inc;
      __syncthreads();
      Sum from = base + inc - mine, all = 0;
      for (int i = 0; i < kVfWarps; ++i) {
        if (i < warp) from += sh.warps[i];
        all += sh.warps[i];
      }
      if (from <= at && at < from + mine) {  // one thread
        int i = 0;
        for (; i < 3 && at >= from + m[i]; ++i) from += m[i];
        a.out[t] = z + 4 * tid + i;
      }
      base += all;
      if (at < base) break;
    }
    break;
  }

  if (c != 0) return;
  for (int i = tid; i <= n; i += kVfThreads) {
    if (i < taken) a.out[t0 + i] = __ldcg(a.tokens + t0 + i + 1);
    if (i > taken) a.out[t0 + i] = -1;
  }
  if (tid == 0) {
    a.accepted[r] = taken;
    if (a.kept) a.kept[r] = __ldcg(a.kv_len + r) - (n - taken);
  }
}

template <class TT, class DT, class Sum>
static cudaError_t launch_vf_sum(const VerifyArgs& a, cudaStream_t s) {
  // as many CTAs a request as there are SMs for (four an SM), where several of more than 1024 tokens each
  unsigned C = 1;
  while (C < unsigned(kVfMost) && int64_t(a.n_req) * C * 2 <= 4 * sm_count() && a.vocab > int64_t(C) * 2048) C *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(a.n_req) * C);
  cfg.blockDim = dim3(kVfThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<TT, DT, Sum>, a);
}

template <class TT, class DT>
static cudaError_t launch_vf(const VerifyArgs& a, cudaStream_t s) {
  return a.vocab < kVfWide ? launch_vf_sum<TT, DT, unsigned long long>(a, s) : launch_vf_sum<TT, DT, unsigned __int128>(a, s);
}

cudaError_t launch_verify_drafts(const VerifyArgs& a, gsi_dtype tdt, gsi_dtype ddt, cudaStream_t s) {
  if (tdt == GSI_F32) return ddt == GSI_F32 ? launch_vf<F32, F32>(a, s) : launch_vf<F32, BF16>(a, s);
  return ddt == GSI_F32 ? launch_vf<BF16, F32>(a, s) : launch_vf<BF16, BF16>(a, s);
}

}  // namespace gsi
