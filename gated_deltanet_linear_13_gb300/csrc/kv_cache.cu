// The paged key/value cache of the full-attention layers: tokens written into it (quantised as
// they are written when the cache holds 8-bit codes) and read back.
//
// 8-bit format: a vector of d elements (one token, one head, keys or values) is stored as e4m3
// codes c with one power-of-two scale 2^e, e the least whole number of [-60, 60] with
// max|x| 2^-e <= 448 (the largest e4m3 value) over the vector's finite elements, and
// c = rne(x 2^-e), saturating.  A power of two costs e4m3 nothing (the format has its own
// exponent, and elements down to max|x| 2^-14 keep all four significant bits), makes scaling
// exact, and every stored value c 2^e is exact in bf16, so reading back rounds nothing.  From
// max|x| = f 2^x, 1 <= f < 2: e = x - 8 when f <= 1.75 (448 = 1.75 2^8), else x - 7.
//
// Both kernels move 16 bytes of the 16-bit side a lane, d / 8 lanes a vector, and are bound by
// memory.
#include <cuda_fp8.h>

#include "common.cuh"

using namespace gdn;

static __device__ unsigned int g_err_kv;

unsigned gdn_take_error_kv_cache() {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_kv, sizeof(v));
  cudaMemcpyToSymbol(g_err_kv, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -60, kMaxExp = 60;

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

__device__ __forceinline__ int scale_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

// Vector index -> (token, keys or values, head): heads fastest, then keys / values, then tokens.
struct Where {
  int token, head, which;
};
__device__ __forceinline__ Where where(long long vec, int H) {
  const long long r = vec / H;
  return Where{(int)(r >> 1), (int)(vec - r * H), (int)(r & 1)};
}

// Element offset of a cache vector, or -1: skipped (negative slot) or out of range (recorded).
__device__ __forceinline__ long long row_of(int slot, int head, int H, int page_shift,
                                            int num_pages) {
  if (slot < 0) return -1;
  const int page = slot >> page_shift, off = slot & ((1 << page_shift) - 1);
  if (page >= num_pages) {
    atomicOr(&g_err_kv, kErrIndex);
    return -1;
  }
  return ((((long long)page * H + head) << page_shift) + off);
}

template <typename Tin, int D, bool kF8>
__global__ void __launch_bounds__(kThreads) gdn_kv_append_kernel(
    GdnKvCacheArgs c, int n, const Tin* k, long long k_stride, const Tin* v, long long v_stride,
    const int32_t* slots) {
  constexpr int L = D / 8;                             // lanes a vector
  const int lane = threadIdx.x % L;
  const long long vecs = 2ll * n * c.H;
  const long long step = (long long)gridDim.x * (kThreads / L);
  // whole warps stay in the loop for the shuffles: past the end, the last vector once more
  const long long first = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  for (long long v0 = first; __any_sync(0xffffffffu, v0 < vecs); v0 += step) {
    const long long vec = v0 < vecs ? v0 : vecs - 1;
    const Where w = where(vec, c.H);
    const long long row =
        v0 < vecs ? row_of(slots[w.token], w.head, c.H, c.page_shift, c.num_pages) : -1;
    const Tin* src = (w.which ? v + w.token * v_stride : k + w.token * k_stride) +
                     (long long)w.head * D + lane * 8;
    const Vec8 x = load8(src);
    if constexpr (!kF8) {
      if (row >= 0)
        store8(static_cast<__nv_bfloat16*>(w.which ? c.v : c.k) + row * D + lane * 8, x);
    } else {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x.x[i]);
        top = m < INFINITY ? fmaxf(top, m) : top;      // false for NaN too
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = scale_exponent(top);
      const float f = pow2i(-e);
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lo |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x.x[2 * i] * f, x.x[2 * i + 1] * f),
                                                 __NV_SATFINITE, __NV_E4M3)
              << (16 * i);
        hi |= (uint32_t)__nv_cvt_float2_to_fp8x2(
                  make_float2(x.x[4 + 2 * i] * f, x.x[5 + 2 * i] * f), __NV_SATFINITE, __NV_E4M3)
              << (16 * i);
      }
      if (row >= 0) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(w.which ? c.v : c.k) + row * D +
                                  lane * 8) = make_uint2(lo, hi);
        if (lane == 0) (w.which ? c.v_exp : c.k_exp)[row] = (uint8_t)(e + 127);
      }
    }
  }
}

template <typename Tout, int D, bool kF8>
__global__ void __launch_bounds__(kThreads) gdn_kv_read_kernel(GdnKvCacheArgs c, int n,
                                                               const int32_t* slots, Tout* k_out,
                                                               Tout* v_out) {
  constexpr int L = D / 8;
  const int lane = threadIdx.x % L;
  const long long vecs = 2ll * n * c.H;
  const long long step = (long long)gridDim.x * (kThreads / L);
  for (long long vec = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L; vec < vecs;
       vec += step) {
    const Where w = where(vec, c.H);
    const long long row = row_of(slots[w.token], w.head, c.H, c.page_shift, c.num_pages);
    Vec8 x = {};
    if (row >= 0) {
      if constexpr (!kF8) {
        x = load8(static_cast<const __nv_bfloat16*>(w.which ? c.v : c.k) + row * D + lane * 8);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(
            static_cast<const uint8_t*>(w.which ? c.v : c.k) + row * D + lane * 8);
        const float f = pow2i((int)(w.which ? c.v_exp : c.k_exp)[row] - 127);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = ((i < 2 ? u.x : u.y) >> (16 * (i & 1))) & 0xffffu;
          const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
          x.x[2 * i] = __low2float(h) * f;
          x.x[2 * i + 1] = __high2float(h) * f;
        }
      }
    }
    store8((w.which ? v_out : k_out) + ((long long)w.token * c.H + w.head) * D + lane * 8, x);
  }
}

int grid_for(long long vecs, int D) {
  const long long blocks = (vecs * (D / 8) + kThreads - 1) / kThreads;
  return (int)(blocks < 152 * 8 ? blocks : 152 * 8);
}

template <typename Tin, int D>
void launch_append(const GdnKvCacheArgs& c, int n, const void* k, long long ks, const void* v,
                   long long vs, const int32_t* slots, cudaStream_t stream) {
  const int grid = grid_for(2ll * n * c.H, D);
  if (c.f8)
    gdn_kv_append_kernel<Tin, D, true><<<grid, kThreads, 0, stream>>>(
        c, n, (const Tin*)k, ks, (const Tin*)v, vs, slots);
  else
    gdn_kv_append_kernel<Tin, D, false><<<grid, kThreads, 0, stream>>>(
        c, n, (const Tin*)k, ks, (const Tin*)v, vs, slots);
}

template <typename Tout, int D>
void launch_read(const GdnKvCacheArgs& c, int n, const int32_t* slots, void* k, void* v,
                 cudaStream_t stream) {
  const int grid = grid_for(2ll * n * c.H, D);
  if (c.f8)
    gdn_kv_read_kernel<Tout, D, true><<<grid, kThreads, 0, stream>>>(c, n, slots, (Tout*)k, (Tout*)v);
  else
    gdn_kv_read_kernel<Tout, D, false><<<grid, kThreads, 0, stream>>>(c, n, slots, (Tout*)k, (Tout*)v);
}

}  // namespace

cudaError_t gdn_launch_kv_append(const GdnKvCacheArgs& c, int n, int in_bf16, const void* k,
                                 long long k_stride, const void* v, long long v_stride,
                                 const int32_t* slots, cudaStream_t stream) {
  if (c.D == 128) {
    if (in_bf16) launch_append<__nv_bfloat16, 128>(c, n, k, k_stride, v, v_stride, slots, stream);
    else launch_append<float, 128>(c, n, k, k_stride, v, v_stride, slots, stream);
  } else {
    if (in_bf16) launch_append<__nv_bfloat16, 256>(c, n, k, k_stride, v, v_stride, slots, stream);
    else launch_append<float, 256>(c, n, k, k_stride, v, v_stride, slots, stream);
  }
  return cudaGetLastError();
}

cudaError_t gdn_launch_kv_read(const GdnKvCacheArgs& c, int n, const int32_t* slots, int out_bf16,
                               void* k_out, void* v_out, cudaStream_t stream) {
  if (c.D == 128) {
    if (out_bf16) launch_read<__nv_bfloat16, 128>(c, n, slots, k_out, v_out, stream);
    else launch_read<float, 128>(c, n, slots, k_out, v_out, stream);
  } else {
    if (out_bf16) launch_read<__nv_bfloat16, 256>(c, n, slots, k_out, v_out, stream);
    else launch_read<float, 256>(c, n, slots, k_out, v_out, stream);
  }
  return cudaGetLastError();
}
