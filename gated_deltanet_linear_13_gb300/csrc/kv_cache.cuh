// What the kernels that write or read the paged key/value cache share: eight elements of a vector
// a lane, and the 8-bit format (see kv_cache.cu).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace gdn {

constexpr int kKvMinExp = -60, kKvMaxExp = 60;

struct Vec8 {
  float x[8];
};

__device__ __forceinline__ Vec8 load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Vec8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.x[2 * i] = __uint_as_float(w[i] << 16);
    v.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return v;
}
__device__ __forceinline__ Vec8 load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Vec8& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const Vec8& v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}

// 2^e for a whole e of [-126, 127]
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ int kv_scale_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kKvMinExp), kKvMaxExp);
}

// Row of a token's slot in the cache (of H * page rows a page), or -1: skipped (negative slot) or
// out of range (recorded in the error word).
__device__ __forceinline__ long long kv_row_of(unsigned int* word, const GdnKvCacheArgs& c, int slot,
                                               int head) {
  if (slot < 0) return -1;
  const int page = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
  if (page >= c.num_pages) {
    atomicOr(word, kErrIndex);
    return -1;
  }
  const long long row = (((long long)page * c.H + head) << c.page_shift) + off;
  return in_bounds(word, head < c.H && row < ((long long)c.num_pages * c.H << c.page_shift))
             ? row
             : -1;
}

// The largest finite size among eight elements (0: none).
__device__ __forceinline__ float kv_largest(const Vec8& v) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float m = fabsf(v.x[e]);
    top = m < INFINITY ? fmaxf(top, m) : top;          // false for NaN too
  }
  return top;
}
// The e4m3 codes of four elements under the scale 2^e.
__device__ __forceinline__ uint32_t kv_codes4(const float* x, int e) {
  const float f = pow2i(-e);
  uint32_t w = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q)
    w |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[2 * q] * f, x[2 * q + 1] * f),
                                            __NV_SATFINITE, __NV_E4M3)
         << (16 * q);
  return w;
}
__device__ __forceinline__ uint2 kv_codes(const Vec8& v, int e) {
  return make_uint2(kv_codes4(v.x, e), kv_codes4(v.x + 4, e));
}

}  // namespace gdn
