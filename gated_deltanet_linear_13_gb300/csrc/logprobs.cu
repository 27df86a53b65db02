// Log probabilities of given tokens with entropy and top alternatives.  First form: one CTA a
// row, the statistics in one pass and each alternative in a pass of its own.
#include "common.cuh"

using namespace gdn;

static __device__ unsigned int g_err_lp;

unsigned gdn_take_error_logprobs() {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_lp, sizeof(v));
  cudaMemcpyToSymbol(g_err_lp, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kThreads = 512;

// Statistics of a set of logits x: maximum m, z = sum e^(x-m), w = sum e^(x-m) (x-m).
struct Stats {
  float m, z, w;
};

__device__ __forceinline__ Stats merge(const Stats& a, const Stats& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY || a.z != a.z || b.z != b.z) return Stats{m, a.z + b.z, a.w + b.w};
  const float da = a.m - m, db = b.m - m;
  const float fa = expf(da), fb = expf(db);
  Stats r{m, 0.0f, 0.0f};
  // a side that underflows adds nothing (its da may be infinite)
  if (fa != 0.0f) r.z += fa * a.z, r.w += fa * (a.w + da * a.z);
  if (fb != 0.0f) r.z += fb * b.z, r.w += fb * (b.w + db * b.z);
  return r;
}

// The order of the alternatives: larger values first (NaN above all, -0 equal to 0), then lower
// indices; packed so that a larger key comes first.
__device__ __forceinline__ unsigned long long order_key(float x, int i) {
  uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
  u = x != x ? 0xffffffffu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((unsigned long long)u << 32) | (uint32_t)~i;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gdn_token_logprobs_simple(GdnLogprobArgs a) {
  __shared__ Stats s_stats[kThreads];
  __shared__ unsigned long long s_key[kThreads];
  const int r = blockIdx.x, t = threadIdx.x;
  const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
  Stats st{-INFINITY, 0.0f, 0.0f};
  bool nan = false;
  for (int i = t; i < a.V; i += kThreads) {
    const float v = ld_elem(x + i) * a.scale;
    if (v != v) nan = true;
    if (v != -INFINITY) st = merge(st, Stats{v, 1.0f, 0.0f});
  }
  if (nan) st.z = NAN;
  s_stats[t] = st;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (t < o) s_stats[t] = merge(s_stats[t], s_stats[t + o]);
    __syncthreads();
  }
  st = s_stats[0];
  const bool dead = st.m == -INFINITY && st.z == 0.0f;
  const float logz = logf(st.z);
  if (t == 0) {
    if (a.logprobs) {
      const int id = a.targets[r];
      float lp = 0.0f;
      if (id >= a.V) {
        atomicOr(&g_err_lp, kErrIndex);
        lp = NAN;
      } else if (id >= 0) {
        lp = dead ? -INFINITY : (ld_elem(x + id) * a.scale - st.m) - logz;
      }
      a.logprobs[r] = lp;
    }
    if (a.entropy) a.entropy[r] = dead ? 0.0f : logz - st.w / st.z;
  }
  unsigned long long below = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    unsigned long long best = 0;
    for (int i = t; i < a.V; i += kThreads) {
      const unsigned long long key = order_key(ld_elem(x + i), i);
      if (key < below && key > best) best = key;
    }
    __syncthreads();
    s_key[t] = best;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
      if (t < o && s_key[t + o] > s_key[t]) s_key[t] = s_key[t + o];
      __syncthreads();
    }
    below = s_key[0];
    if (t == 0) {
      const int id = (int)~(uint32_t)below;
      a.top_ids[(long long)r * a.top_k + k] = id;
      a.top_logprobs[(long long)r * a.top_k + k] =
          dead ? -INFINITY : (ld_elem(x + id) * a.scale - st.m) - logz;
    }
  }
}

}  // namespace

size_t gdn_token_logprobs_bytes(int, int, int, int) { return 0; }

cudaError_t gdn_launch_token_logprobs(const GdnLogprobArgs& a, cudaStream_t stream) {
  if (a.bf16) gdn_token_logprobs_simple<__nv_bfloat16><<<a.N, kThreads, 0, stream>>>(a);
  else gdn_token_logprobs_simple<float><<<a.N, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
