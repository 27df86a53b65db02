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
// Both kernels move eight elements a lane, d / 8 lanes a vector, four tokens of a lane on the way
// at a time (one: 29.4 and 51.9 us below), and are bound by memory: 16384 bf16 tokens of 4 x 256
// into an 8-bit cache 19.4 us (5.2 TB/s read and written), 40001 tokens of 8 x 128 out of one
// 42.7 us (5.8 TB/s); a few tokens cost one launch, 2.2 us.
#include "common.cuh"
#include "kv_cache.cuh"

using namespace gdn;

static __device__ unsigned int g_err_kv;

unsigned gdn_take_error_kv_cache() { return gdn::take_error(g_err_kv); }

namespace {

constexpr int kThreads = 256;

// Grid: x tokens, y = keys of head 0 .. H - 1, then values.  d / 8 lanes a vector; a thread has
// kTokens tokens, kThreads 8 / d apart, their loads issued before any use.
constexpr int kTokens = 4;

template <typename Tin, int D, bool kF8>
__global__ void __launch_bounds__(kThreads) gdn_kv_append_kernel(
    GdnKvCacheArgs c, int n, const Tin* k, long long k_stride, const Tin* v, long long v_stride,
    const int32_t* slots) {
  constexpr int L = D / 8, kStep = kThreads / L;
  const int lane = threadIdx.x % L;
  const bool values = (int)blockIdx.y >= c.H;
  const int head = values ? blockIdx.y - c.H : blockIdx.y;
  const long long stride = values ? v_stride : k_stride;
  const Tin* src = (values ? v : k) + (long long)head * D + lane * 8;
  const int t0 = blockIdx.x * (kStep * kTokens) + threadIdx.x / L;
  int slot[kTokens];
  Vec8 x[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int t = t0 + i * kStep;
    slot[i] = t < n && in_bounds(&g_err_kv, t >= 0) ? slots[t] : -1;
    x[i] = load8(src + min(t, n - 1) * stride);       // (whole warps stay for the shuffles)
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    long long row = kv_row_of(&g_err_kv, c, slot[i], head);
    if (!in_bounds(&g_err_kv, head >= 0 && lane * 8 + 8 <= D)) row = -1;
    if constexpr (!kF8) {
      if (row >= 0) store8(static_cast<__nv_bfloat16*>(values ? c.v : c.k) + row * D + lane * 8, x[i]);
    } else {
      float top = kv_largest(x[i]);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = kv_scale_exponent(top);
      const uint2 codes = kv_codes(x[i], e);
      if (row >= 0) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(values ? c.v : c.k) + row * D + lane * 8) =
            codes;
        if (lane == 0) (values ? c.v_exp : c.k_exp)[row] = (uint8_t)(e + 127);
      }
    }
  }
}

template <typename Tout, int D, bool kF8>
__global__ void __launch_bounds__(kThreads) gdn_kv_read_kernel(GdnKvCacheArgs c, int n,
                                                               const int32_t* slots, Tout* k_out,
                                                               Tout* v_out) {
  constexpr int L = D / 8, kStep = kThreads / L;
  const int lane = threadIdx.x % L;
  const bool values = (int)blockIdx.y >= c.H;
  const int head = values ? blockIdx.y - c.H : blockIdx.y;
  const int t0 = blockIdx.x * (kStep * kTokens) + threadIdx.x / L;
  long long row[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int t = t0 + i * kStep;
    row[i] = kv_row_of(&g_err_kv, c, t < n && in_bounds(&g_err_kv, t >= 0) ? slots[t] : -1, head);
  }
  Vec8 x[kTokens];
  if constexpr (!kF8) {
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(values ? c.v : c.k) + lane * 8;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) x[i] = row[i] >= 0 ? load8(base + row[i] * D) : Vec8{};
  } else {
    const uint8_t* base = static_cast<const uint8_t*>(values ? c.v : c.k) + lane * 8;
    const uint8_t* exps = values ? c.v_exp : c.k_exp;
    uint2 u[kTokens];
    int e[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      u[i] = row[i] >= 0 ? *reinterpret_cast<const uint2*>(base + row[i] * D) : make_uint2(0, 0);
      e[i] = row[i] >= 0 ? exps[row[i]] : 127;
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const float f = __uint_as_float((uint32_t)e[i] << 23);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t two = ((q < 2 ? u[i].x : u[i].y) >> (16 * (q & 1))) & 0xffffu;
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
        x[i].x[2 * q] = __low2float(h) * f;
        x[i].x[2 * q + 1] = __high2float(h) * f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int t = t0 + i * kStep;
    if (t < n && in_bounds(&g_err_kv, t >= 0 && head < c.H && lane * 8 + 8 <= D))
      store8((values ? v_out : k_out) + ((long long)t * c.H + head) * D + lane * 8, x[i]);
  }
}

dim3 grid_for(int n, int H, int D) {
  const int tokens = kThreads / (D / 8) * kTokens;
  return dim3((unsigned)((n + (long long)tokens - 1) / tokens), (unsigned)(2 * H));
}

template <typename Tin, int D>
void launch_append(const GdnKvCacheArgs& c, int n, const void* k, long long ks, const void* v,
                   long long vs, const int32_t* slots, cudaStream_t stream) {
  const dim3 grid = grid_for(n, c.H, D);
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
  const dim3 grid = grid_for(n, c.H, D);
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

// One error word a translation unit, and reading it is the error query's time (9 us a word): the
// operators around the cache share its.
#include "pages.cuh"
#include "qk_norm_rope.cuh"
