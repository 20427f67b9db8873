// Attention of new tokens over a paged key/value cache: dispatch, and the
// plain kernel.

#include <algorithm>

#include "gsi_attn.cuh"

namespace gsi {

// The plain kernel, for more than 64 heads of a float32 model that share a
// key/value head (its row tiles hold 64 rows): one warp a (token, head), the
// running maximum m and sum l of a softmax and its weighted sum o over the
// row's keys, one pass,
//   m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') + e^(s - m') v,
// 32 keys at a time (a lane scores one key; the weighted sum has the lanes on
// the head's columns).
constexpr int kPlainWarps = 4;

template <class T>
__global__ void __launch_bounds__(kPlainWarps * 32) attn_plain_kernel(AttnArgs a) {
  __shared__ float s_q[kPlainWarps][256];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * kPlainWarps + warp;
  const int hq = a.hkv * a.group;
  const int64_t tok = w / hq;
  const int head = int(w - tok * hq);
  if (tok >= a.N) return;
  // its request: the last one that begins at or before the token
  int lo = 0, hi = a.n_req;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(a.q_start + mid) <= tok) lo = mid; else hi = mid;
  }
  const int r = lo;
  const int64_t q0 = __ldcg(a.q_start + r), q1 = __ldcg(a.q_start + r + 1);
  if (tok < q0 || tok >= q1) return;
  const int64_t most = a.width << a.page_shift;
  const int64_t len = min(max(int64_t(__ldcg(a.kv_len + r)), int64_t(0)), most);
  const int64_t lim = a.causal ? max(int64_t(0), len - (q1 - tok) + 1) : len;
  const int64_t first = a.window > 0 ? max(int64_t(0), lim - a.window) : 0;
  for (int c = lane; c < a.dim; c += 32) s_q[warp][c] = T::load1_cg(a.Q, tok * a.q_stride + int64_t(head) * a.dim + c) * a.scale;
  __syncwarp();
  const int kvh = head / a.group;
  float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  for (int64_t j0 = first; j0 < lim; j0 += 32) {
    const int64_t j = j0 + lane;
    float s = -INFINITY;
    int64_t at = -1;
    if (j < lim) {
      const int64_t pg = __ldcg(a.table + r * a.width + (j >> a.page_shift));
      s = 0.f;
      if (pg >= 0 && pg < a.n_pages) {
        at = pg * a.page_stride + kvh * a.head_stride + (j & ((1 << a.page_shift) - 1)) * a.token_stride;
        for (int c = 0; c < a.dim; ++c) s = fmaf(s_q[warp][c], T::load1_cg(a.K, at + c), s);
      }
    }
    float mx = s;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    mx = fmaxf(mx, m);
    const float p = j < lim ? (s == -INFINITY ? 0.f : expf(s - mx)) : 0.f;
    const float f = m == -INFINITY ? 0.f : expf(m - mx);
    m = mx;
    l = l * f + warp_sum(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= f;
    const int n = int(min(int64_t(32), lim - j0));
    for (int k = 0; k < n; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      const int64_t ak = __shfl_sync(0xffffffffu, (long long)at, k);
      if (ak >= 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = lane + 32 * i;
          if (c < a.dim) o[i] = fmaf(pk, T::load1_cg(a.V, ak + c), o[i]);
        }
    }
  }
  const float inv = l != 0.f ? 1.f / l : lim > 0 ? NAN : 0.f;  // as attn_inverse
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = lane + 32 * i;
    if (c < a.dim) T::store1(a.O, (tok * hq + head) * a.dim + c, o[i] * inv);
  }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*AttnEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static AttnEncodeFn attn_encode_fn() {
  static const AttnEncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess && q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<AttnEncodeFn>(p) : nullptr;
  }();
  return fn;
}

cudaError_t attn_page_map(CUtensorMap* m, const AttnArgs& a, const void* base, int box_rows) {
  const AttnEncodeFn fn = attn_encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t page = cuuint64_t(1) << a.page_shift;
  cuuint64_t dim[4] = {cuuint64_t(a.dim), page, cuuint64_t(a.hkv), cuuint64_t(a.n_pages)};
  // the stride of a dimension of one element is never used: any valid one does
  const int64_t st[3] = {a.token_stride, a.hkv > 1 ? a.head_stride : a.token_stride,
                         a.n_pages > 1 ? a.page_stride : a.token_stride};
  cuuint64_t bytes[3];
  for (int i = 0; i < 3; ++i) bytes[i] = cuuint64_t(st[i]) * 2;
  if (a.n_pages == 0) {  // nothing is read through it (no request then has a key)
    base = a.Q;
    dim[1] = dim[2] = dim[3] = 1;
  }
  const cuuint32_t box[4] = {64, cuuint32_t(box_rows), 1, 1}, es[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dim, bytes, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t attn_query_map(CUtensorMap* m, const AttnArgs& a, int box_heads, int box_tokens) {
  const AttnEncodeFn fn = attn_encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dim[3] = {cuuint64_t(a.dim), cuuint64_t(a.hkv) * a.group, cuuint64_t(a.N)};
  const cuuint64_t bytes[2] = {cuuint64_t(a.dim) * 2, cuuint64_t(a.q_stride) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)}, es[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.Q), dim, bytes, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int sm_count() {
  static std::atomic<int> counts[64];
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return kAttnCtas;
  if ((v = counts[dev].load(std::memory_order_relaxed)) > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return kAttnCtas;
  counts[dev].store(v, std::memory_order_relaxed);
  return v;
}

size_t attention_work_bytes(gsi_dtype dt, int dim, int group) {
  return dt == GSI_BF16 ? attn_tiles_work_bytes(dim) : attn_work_bytes(2 * kAttnCtas, 64, dim);
}

// Few query rows of a request under one key/value head go to the kernels of 8
// (float32: 16) rows, which the bytes bound; more to the row tiles.  Both sides,
// us: bf16, 8 heads that share one of 8 key/value heads of 128 columns, 2000 keys
// 14.4 (row tiles 14.8), 8 requests of 8000 keys 41 (44); 16 heads 19 (16) and 53
// (45).  float32, 16 rows over 2000 keys of 8 x 64: 31 (44); 32 rows 43 (47).
constexpr int64_t kF32FewTiles = 304;
cudaError_t launch_paged_attention(const AttnArgs& a, gsi_dtype dt, int64_t max_q, cudaStream_t s) {
  // The hint is the caller's: a request that has tokens has at least one and no more than all of them, whatever it says
  // (a unit of the few-row kernels has to hold a token's heads).
  const int64_t most = std::clamp<int64_t>(max_q, 1, a.N) * a.group;
  if (dt == GSI_BF16) return most <= 8 ? launch_attn_rows(a, s) : launch_attn_tiles(a, s);
  if (a.group <= 64) {
    // 64-row units that do not fill the chip are too long a chain each.  `tiles` is what their tiles would be if rows filled
    // them: an estimate, which leaves out each request's part of a unit (whose empty rows the 16-row units save).  16 and 64
    // rows, us: 64 tokens, window 128, 4 x 64 16 and 24; 100 of 500, 4 requests of 4 x 64 27 and 29; 17 of 500, 100 requests of
    // 1 x 64 26 and 36; 17 of 2000, 24 requests 26 and 35; but 17 of 500, 60 requests 25 and 22; and beyond the rule's bound
    // 100 of 1000, 4 requests of 8 / 4 x 128 77 and 71, 128 of 1000, 8 requests of 8 x 64 90 and 62, 60 of 800, 6 requests of
    // 8 / 2 x 32 33 and 22, 64 of 500, 16 requests of 4 / 2 x 128 43 and 47
    const int64_t keys = std::min<int64_t>(a.width << a.page_shift, a.window > 0 ? int64_t(a.window) + 128 : int64_t(1) << 31);
    const int64_t tiles = (int64_t(a.N) * a.group / 64 + 1) * a.hkv * (keys / 64 + 1);
    return launch_attn_f32(a, most <= 16 || (a.group <= 16 && tiles < kF32FewTiles), s);
  }
  const int64_t rows = int64_t(a.N) * a.hkv * a.group;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned((rows + kPlainWarps - 1) / kPlainWarps));
  cfg.blockDim = dim3(kPlainWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_plain_kernel<F32>, a);
}

}  // namespace gsi
