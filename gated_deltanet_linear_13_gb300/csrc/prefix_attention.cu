// Attention of a batch that shares a long prefix, over the paged key/value cache.  First form:
// one warp a query row, keys one after the other with a running maximum and sum.
#include <cuda_fp8.h>

#include "common.cuh"

using namespace gdn;

static __device__ unsigned int g_err_attn;

unsigned gdn_take_error_prefix_attention() {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_attn, sizeof(v));
  cudaMemcpyToSymbol(g_err_attn, &z, sizeof(z));
  return v;
}

namespace {

template <int D, bool kF8>
__device__ __forceinline__ void load_row(const void* base, const uint8_t* exps, long long row,
                                         int lane, float (&x)[D / 32]) {
  constexpr int E = D / 32;
  if constexpr (kF8) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + row * D + lane * E;
    const float f = exp2f((float)exps[row] - 127.0f);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const __half h = __half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3));
      x[i] = __half2float(h) * f;
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + row * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __bfloat162float(p[i]);
  }
}

template <int D, bool kF8, typename Tout>
__global__ void __launch_bounds__(128) gdn_prefix_attention_simple(GdnAttnArgs a) {
  constexpr int E = D / 32;
  const GdnKvCacheArgs& c = a.cache;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.T * a.Hq) return;
  const int tok = (int)(row / a.Hq), hq = (int)(row % a.Hq), h = hq / (a.Hq / c.H);
  const int b = tok / a.T, t = tok % a.T;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.0f;
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + tok * a.q_stride +
                            (long long)hq * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) q[i] = __bfloat162float(qp[i]);
  int len = a.kv_len[b];
  const bool active = len >= 0;
  const long long most = (long long)a.max_pages << c.page_shift;
  if (len > most) {
    if (lane == 0) atomicOr(&g_err_attn, kErrIndex);
    len = (int)most;
  }
  const int own = max(0, min(len, len - a.T + 1 + t));
  const int pm = (1 << c.page_shift) - 1;
  const long long total = active ? (long long)a.prefix_len + own : 0;
  for (long long j = 0; j < total; ++j) {
    const bool pre = j < a.prefix_len;
    const int i = (int)(pre ? j : j - a.prefix_len);
    const int page = pre ? a.prefix_pages[i >> c.page_shift]
                         : a.pages[(long long)b * a.max_pages + (i >> c.page_shift)];
    float k[E] = {}, v[E] = {};
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) atomicOr(&g_err_attn, kErrIndex);
    } else {
      const long long r = (((long long)page * c.H + h) << c.page_shift) + (i & pm);
      load_row<D, kF8>(c.k, c.k_exp, r, lane, k);
      load_row<D, kF8>(c.v, c.v_exp, r, lane, v);
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s) * a.scale;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.0f : mn;
    const float f = expf(m - base), p = expf(s - base);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * v[e];
  }
  Tout* op = static_cast<Tout*>(a.out) + row * D + lane * E;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) st_elem(op + e, o[e] * inv);
  if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <int D, bool kF8>
void launch(const GdnAttnArgs& a, cudaStream_t stream) {
  const long long rows = (long long)a.B * a.T * a.Hq;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  if (a.out_bf16) gdn_prefix_attention_simple<D, kF8, __nv_bfloat16><<<grid, 128, 0, stream>>>(a);
  else gdn_prefix_attention_simple<D, kF8, float><<<grid, 128, 0, stream>>>(a);
}

}  // namespace

size_t gdn_prefix_attention_bytes(int, int, int, int, int) { return 0; }

cudaError_t gdn_launch_prefix_attention(const GdnAttnArgs& a, cudaStream_t stream) {
  if (a.cache.D == 128) {
    if (a.cache.f8) launch<128, true>(a, stream);
    else launch<128, false>(a, stream);
  } else {
    if (a.cache.f8) launch<256, true>(a, stream);
    else launch<256, false>(a, stream);
  }
  return cudaGetLastError();
}
