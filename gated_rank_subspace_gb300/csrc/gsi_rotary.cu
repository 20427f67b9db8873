// Rotary positions: the angles' table (host), and the append of a qkv map's rows
// whose queries and keys are turned by them.

#include <cmath>

#include "gsi_append.cuh"
#include "gsi_kernels.h"

namespace gsi {

// Pair i of a head, (a, b), at position p turns by the angle p w_i:
//   a' = s (a cos - b sin),  b' = s (b cos + a sin)
// with (a, b) the values (2 i, 2 i + 1) or (i, turned / 2 + i).  An angle of
// many turns has no fraction left in 32 bits (position 10^6 and w = 1: 0.06), so
// a rate is kept as the fraction of a turn a position adds, in units of 2^-64:
// p times it, modulo 2^64, is the fraction of a turn that p adds, exactly, by
// one integer product.  Its nearest quarter turn is taken off, and what is left
// (under an eighth) becomes a float32 with all its bits.
//
// A copy otherwise: the bytes bound it, and a CTA's chain position, angle, barrier
// (2048 tokens of 16 + 2 x 16 heads of 256 29 us, 5.2 TB/s; the plain append 24).  A
// CTA takes a token, or 512 16-byte output vectors of it where tokens are few, and
// forms the token's sines and cosines once, in shared memory.  With values i and turned / 2 + i, one thread makes both output
// vectors where they are aligned, so that each row is read once.
constexpr int kRotaryThreads = 256;

__device__ __forceinline__ float2 rotary_turn(unsigned long long rate, int64_t pos, float scale) {
  const int32_t turn = int32_t((uint64_t(pos) * rate) >> 32);  // 2^-32 of a turn
  const int32_t quarter = int32_t((uint32_t(turn) + 0x20000000u) >> 30) & 3;
  const int32_t rest = int32_t(uint32_t(turn) - (uint32_t(quarter) << 30));  // within an eighth of a turn
  float s, c;
  sincospif(float(rest) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  s *= scale;
  c *= scale;
  return quarter == 0 ? make_float2(c, s) : quarter == 1 ? make_float2(-s, c) : quarter == 2 ? make_float2(-c, -s) : make_float2(s, -c);
}

// N values of a row from element e on: as they are, and as float32.
template <class XT, int N>
struct RotaryValues {
  static constexpr int kBytes = N * XT::kBytes;
  uint4 v[(kBytes + 15) / 16];
  __device__ __forceinline__ void load(const char* row, int64_t e) {
    if constexpr (kBytes == 8) {  // four bf16 values for a float32 vector
      const uint2 u = __ldcg(reinterpret_cast<const uint2*>(row + e * XT::kBytes));
      v[0] = make_uint4(u.x, u.y, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) v[i] = ld_cg_v4(row + e * XT::kBytes + 16 * i);
    }
  }
  __device__ __forceinline__ void floats(float (&f)[N]) const {
    if constexpr (kBytes == 8) {
      BF16::unpack2(v[0].x, f[0], f[1]);
      BF16::unpack2(v[0].y, f[2], f[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        float w[XT::kPerVec];
        XT::unpack(v[i], w);
#pragma unroll
        for (int x = 0; x < XT::kPerVec; ++x) f[i * XT::kPerVec + x] = w[x];
      }
    }
  }
};
template <class CT, int N>
__device__ __forceinline__ void rotary_store(char* dst, const float (&f)[N]) {
  if constexpr (CT::kBytes == 2)
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  else
    *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
}

template <class XT, class CT>
__global__ void __launch_bounds__(kRotaryThreads) rotary_append_kernel(const __grid_constant__ RotaryArgs r) {
  constexpr int N = CT::kPerVec;
  __shared__ float2 s_turn[128];
  const AppendArgs& a = r.to;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int half = r.turned / 2;
  if (int(threadIdx.x) < half) {
    int64_t pos = __ldcg(r.positions + t);
    if (r.offsets) {
      const int req = r.token_req ? __ldcg(r.token_req + t) : 0;
      if (req >= 0 && req < r.n_req) pos += __ldcg(r.offsets + req);
    }
    s_turn[threadIdx.x] = rotary_turn(__ldcg(reinterpret_cast<const unsigned long long*>(r.phases) + threadIdx.x), pos, r.scale);
  }
  const int64_t slot = __ldcg(reinterpret_cast<const long long*>(a.slots) + t);
  const bool there = slot >= 0 && slot < a.n_slots;
  const int64_t pg = slot >> a.page_shift, off = slot & ((int64_t(1) << a.page_shift) - 1);
  const int per_head = a.dim / N;
  const int n_vec = (a.hq + 2 * a.hkv) * per_head;
  const char* row = static_cast<const char*>(a.X) + t * a.row_stride * XT::kBytes;
  const bool whole = half % N == 0;  // a vector's partners are a vector
  __syncthreads();
  const int stride = gridDim.y * kRotaryThreads;
#pragma unroll 2
  for (int v = blockIdx.y * kRotaryThreads + threadIdx.x; v < n_vec; v += stride) {
    int head = v / per_head;
    const int e = (v - head * per_head) * N;
    const int64_t first = int64_t(head) * a.dim;  // of the head's values in the row
    const bool turns = head < a.hq + a.hkv && e < r.turned;
    char* dst;
    if (head < a.hq) {
      if (!a.Q) continue;
      dst = static_cast<char*>(a.Q) + ((t * a.hq + head) * a.dim + e) * CT::kBytes;
    } else {
      if (!there) break;
      head -= a.hq;
      const bool val = head >= a.hkv;
      if (val) head -= a.hkv;
      dst = static_cast<char*>(val ? a.V : a.K) + (pg * a.page_stride + head * a.head_stride + off * a.token_stride + e) * CT::kBytes;
    }
    // every lane's loads first: a warp's lanes turn and copy side by side
    const bool halves = turns && !r.pairs && whole;
    if (halves && e >= half) continue;  // made with its partner
    RotaryValues<XT, N> own, partner;
    own.load(row, first + e);
    if (halves) partner.load(row, first + half + e);
    float x[N], y[N];
    own.floats(x);
    if (!turns) {
      if constexpr (XT::kBytes == CT::kBytes)
        *reinterpret_cast<uint4*>(dst) = own.v[0];
      else
        rotary_store<CT, N>(dst, x);
    } else if (r.pairs) {
#pragma unroll
      for (int z = 0; z < N; z += 2) {
        const bool in = e + z < r.turned;
        const float2 cs = in ? s_turn[(e + z) / 2] : make_float2(1.f, 0.f);
        y[z] = in ? fmaf(x[z], cs.x, -x[z + 1] * cs.y) : x[z];
        y[z + 1] = in ? fmaf(x[z + 1], cs.x, x[z] * cs.y) : x[z + 1];
      }
      rotary_store<CT, N>(dst, y);
    } else if (halves) {
      float p[N], q[N];
      partner.floats(p);
#pragma unroll
      for (int z = 0; z < N; ++z) {
        const float2 cs = s_turn[e + z];
        y[z] = fmaf(x[z], cs.x, -p[z] * cs.y);
        q[z] = fmaf(p[z], cs.x, x[z] * cs.y);
      }
      rotary_store<CT, N>(dst, y);
      rotary_store<CT, N>(dst + half * CT::kBytes, q);
    } else {
#pragma unroll
      for (int z = 0; z < N; ++z) {
        const int el = e + z;
        y[z] = x[z];
        if (el < r.turned) {
          const bool low = el < half;
          const float2 cs = s_turn[low ? el : el - half];
          const float p = XT::load1_cg(row, first + (low ? el + half : el - half));
          y[z] = fmaf(x[z], cs.x, (low ? -p : p) * cs.y);
        }
      }
      rotary_store<CT, N>(dst, y);
    }
  }
}

cudaError_t launch_rotary_append(const RotaryArgs& r, gsi_dtype xdt, gsi_dtype cdt, cudaStream_t s) {
  const AppendArgs& a = r.to;
  const int n_vec = (a.hq + 2 * a.hkv) * (a.dim / (cdt == GSI_BF16 ? 8 : 4));
  cudaLaunchConfig_t cfg{};
  // many tokens: a CTA each, which forms its angles once (three CTAs a token of 48 heads of 256 took 32 us for 2048 tokens, one
  // 29); few: spread over the SMs
  const int parts = (n_vec + 2 * kRotaryThreads - 1) / (2 * kRotaryThreads);
  cfg.gridDim = dim3(a.T, a.T >= 2 * sm_count() ? 1 : parts);
  cfg.blockDim = dim3(kRotaryThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (xdt == GSI_F32)
    return cdt == GSI_F32 ? cudaLaunchKernelEx(&cfg, rotary_append_kernel<F32, F32>, r)
                          : cudaLaunchKernelEx(&cfg, rotary_append_kernel<F32, BF16>, r);
  return cdt == GSI_F32 ? cudaLaunchKernelEx(&cfg, rotary_append_kernel<BF16, F32>, r)
                        : cudaLaunchKernelEx(&cfg, rotary_append_kernel<BF16, BF16>, r);
}

// ------------------------------------------------------------------ host side
void rotary_rates(int dim, double base, int scaling, double factor, double context, double fast, double slow, double* rates,
                  float* scale) {
  constexpr double kTurn = 6.283185307179586;
  if (scaling == GSI_ROTARY_NTK) base *= std::pow(factor, dim / (dim - 2.0));
  double low = 0, high = 0;
  if (scaling == GSI_ROTARY_YARN) {
    auto at = [&](double turns) { return dim * std::log(context / (kTurn * turns)) / (2 * std::log(base)); };
    low = std::fmax(0.0, std::floor(at(fast)));
    high = std::fmin(dim - 1.0, std::ceil(at(slow)));
  }
  for (int i = 0; i < dim / 2; ++i) {
    const double w = std::pow(base, -2.0 * i / dim);
    double keep = 1;  // share of the rate that is not divided
    if (scaling == GSI_ROTARY_LINEAR) keep = 0;
    if (scaling == GSI_ROTARY_YARN) keep = 1 - std::fmin(1.0, std::fmax(0.0, (i - low) / std::fmax(high - low, 0.001)));
    if (scaling == GSI_ROTARY_BANDS) keep = std::fmin(1.0, std::fmax(0.0, (context * w / kTurn - slow) / (fast - slow)));
    rates[i] = w * keep + w / factor * (1 - keep);
    if (scaling == GSI_ROTARY_NONE || scaling == GSI_ROTARY_NTK) rates[i] = w;
  }
  *scale = scaling == GSI_ROTARY_YARN ? float(0.1 * std::log(factor) + 1) : 1.f;
}

uint64_t rotary_phase(double rate) {
  // the rate (2^40 at most) over 2 pi as a sum of two doubles: hi, and what its rounding and that of 1 / (2 pi) leave (below
  // 2^-14 of a turn, known to 2^-66)
  constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;  // 1 / (2 pi)
  const double hi = rate * kInv, lo = std::fma(rate, kInv, -hi) + rate * kInvLow;
  // 2^64 (hi - its nearest whole + lo): the difference is exact, and unsigned sums wrap as turns do
  const double a = std::ldexp(hi - std::rint(hi), 64), b = std::rint(std::ldexp(lo, 64));
  const uint64_t ua = a >= 9223372036854775808.0 ? uint64_t(1) << 63 : uint64_t(int64_t(a));
  return ua + uint64_t(int64_t(b));
}

}  // namespace gsi
