// Vectors of a qkv map's rows in the cache's type, for the kernels that store
// them.
#pragma once

#include "gsi_common.cuh"

namespace gsi {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One 16-byte vector of the cache's type from the row's values (float32 to
// bf16 rounds to nearest even; bf16 to float32 is exact).
template <class XT, class CT>
__device__ __forceinline__ uint4 append_vec(const void* row, int64_t e) {
  if constexpr (XT::kBytes == CT::kBytes) {
    return ld_cg_v4(static_cast<const char*>(row) + e * XT::kBytes);
  } else if constexpr (XT::kBytes == 4) {
    const uint4 a = ld_cg_v4(static_cast<const char*>(row) + e * 4), b = ld_cg_v4(static_cast<const char*>(row) + e * 4 + 16);
    return make_uint4(pack_bf16(__uint_as_float(a.x), __uint_as_float(a.y)), pack_bf16(__uint_as_float(a.z), __uint_as_float(a.w)),
                      pack_bf16(__uint_as_float(b.x), __uint_as_float(b.y)), pack_bf16(__uint_as_float(b.z), __uint_as_float(b.w)));
  } else {
    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(static_cast<const char*>(row) + e * 2));
    return make_uint4(v.x << 16, v.x & 0xffff0000u, v.y << 16, v.y & 0xffff0000u);
  }
}

}  // namespace gsi
