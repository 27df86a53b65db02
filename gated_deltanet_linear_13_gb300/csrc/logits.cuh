// Rows of logits as the kernels that go over a vocabulary read them: granules of a kilobyte, a warp's
// at a time, from the 16-byte boundary at or below the row on (rows may start at any element).
#pragma once

#include "common.cuh"

namespace gdn {

template <typename T>
struct Granule {
  static constexpr int kVec = 16 / (int)sizeof(T);     // logits of a 16-byte vector
  static constexpr int kPer = 2 * kVec;                // of a lane
  static constexpr int kLogits = 32 * kPer;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest (NaN if there is one) and the least of two vectors' logits.
__device__ __forceinline__ uint32_t max_word(const uint4& u) {
  return max2_nan(max2_nan(u.x, u.y), max2_nan(u.z, u.w));
}
__device__ __forceinline__ float max_half(uint32_t w) {
  return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void range(const uint4& u, const uint4& v, const __nv_bfloat16*,
                                      const float*, float* top, float* least) {
  *top = max_half(max2_nan(max_word(u), max_word(v)));
  const uint32_t lo =
      min2(min2(min2(u.x, u.y), min2(u.z, u.w)), min2(min2(v.x, v.y), min2(v.z, v.w)));
  *least = fminf(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u));
}
__device__ __forceinline__ void range(const uint4&, const uint4&, const float*, const float* f,
                                      float* top, float* least) {
  *top = max_nan(max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3])),
                 max_nan(max_nan(f[4], f[5]), max_nan(f[6], f[7])));
  *least = fminf(fminf(fminf(f[0], f[1]), fminf(f[2], f[3])),
                 fminf(fminf(f[4], f[5]), fminf(f[6], f[7])));
}
// one vector's largest
__device__ __forceinline__ float vector_top(const uint4& u, const __nv_bfloat16*) {
  return max_half(max_word(u));
}
__device__ __forceinline__ float vector_top(const uint4& u, const float*) {
  return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                 max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
}

__device__ __forceinline__ void widen(const uint4& u, const __nv_bfloat16*, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const uint4& u, const float*, float* x) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
// kOnce: nothing reads it again (its line goes first from L2).
template <bool kOnce = true, typename T>
__device__ __forceinline__ uint4 load_inner(const T* at) {
  uint4 u;
  if constexpr (kOnce)
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(at));
  else
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(at));
  return u;
}

// 16 bytes of logits from the 16-byte boundary at or below row + i on (i: the index of the first,
// which may lie before the row), -inf in the place of what is not the row's.
template <bool kOnce = true, typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, long long i, int V) {
  constexpr int kVec = Granule<T>::kVec;
  if (i >= 0 && i + kVec <= V) return load_inner<kOnce>(row + i);
  uint32_t w[4];
  constexpr int kWord = kVec / 4;                     // logits of a 32-bit word
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w[q] = kWord == 2 ? 0xff80ff80u : 0xff800000u;    // -inf
#pragma unroll
    for (int b = 0; b < kWord; ++b) {
      const long long at = i + q * kWord + b;
      if (at < 0 || at >= V) continue;
      if constexpr (kWord == 1) w[q] = reinterpret_cast<const uint32_t*>(row)[at];
      else
        w[q] = (w[q] & (0xffff0000u >> (16 * b))) |
               (uint32_t)reinterpret_cast<const uint16_t*>(row)[at] << (16 * b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ int shift_of(const T* row) {   // logits from a 16-byte boundary to a row
  return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

inline int granules_of(int V, int bf16) {             // with up to a vector's worth of shift
  const int vec = bf16 ? Granule<__nv_bfloat16>::kVec : Granule<float>::kVec;
  const int per = bf16 ? Granule<__nv_bfloat16>::kLogits : Granule<float>::kLogits;
  return (int)(((long long)V + vec - 1 + per - 1) / per);
}

}  // namespace gdn
