// Log probabilities of given tokens with entropy and top alternatives, in one pass over the
// logits.
//
// Per set of logits x: the maximum m, z = sum 2^t and w = sum 2^t t with t = (x - m) scale log2 e;
// two sets join by rescaling to the larger maximum.  Then logp(i) = (x_i - m) scale - ln z and the
// entropy is ln 2 (log2 z - w / z): centred on m, so that nothing cancels and nothing overflows
// however large the logits are.
//
// The alternatives ride along: a CTA holds a threshold, a lower bound of the k-th best, and only
// logits at or above it go to a buffer in shared memory: almost none after the first ones.  The
// first threshold comes from the threads' maxima over their first logits: the least over the
// CTA's 8 warps of the ceil(k / 8)-th largest of a warp's, which at least k logits reach.  When
// the buffer fills, the best k stay and the k-th is the new threshold.  A logit and its index make
// one 64-bit key, ordered by value (NaN first, -0 equal to 0) and then by lower index; keys are
// distinct, so what is kept does not depend on the order in which threads arrive.
//
// All rows lie on one line of granules (kThreads x 32 bytes, the last of a row shorter); CTA c of
// the grid takes the c-th equal part of it, so one long row fills the GPU as well as a thousand.
// A CTA's piece of a row leaves its statistics and best k; a second, small kernel joins a row's
// pieces.
//
// Bound by memory: each logit is read once.  At the copy rate an SM gets 12 bf16 logits a cycle,
// for which it can issue 128 lane operations; a logit takes about six (packed fp32 pairs where
// there are such instructions) and one of 16 exponentials a cycle.
#include "common.cuh"
#include "sm100_ptx.cuh"

using namespace gdn;

static __device__ unsigned int g_err_lp;

unsigned gdn_take_error_logprobs() {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_lp, sizeof(v));
  cudaMemcpyToSymbol(g_err_lp, &z, sizeof(z));
  return v;
}

namespace {

typedef unsigned long long Key;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4, kCtas = 152 * kCtasPerSm;
constexpr int kBuffer = 1024;              // candidates (of keys) in shared memory
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename T>
struct Granule {
  static constexpr int kVec = 16 / (int)sizeof(T);     // logits of a 16-byte vector
  static constexpr int kPer = 2 * kVec;                // of a thread
  static constexpr int kLogits = kThreads * kPer;
};

// m = -inf: no logit above -inf.  A NaN among the logits: z is NaN.
struct Stats {
  float m, z, w;
};

__device__ __forceinline__ Stats merge(const Stats& a, const Stats& b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY || a.z != a.z || b.z != b.z) return Stats{m, a.z + b.z, a.w + b.w};
  const float da = (a.m - m) * c, db = (b.m - m) * c;
  const float fa = ptx::ex2_approx(da), fb = ptx::ex2_approx(db);
  Stats r{m, 0.0f, 0.0f};
  // a side that underflows adds nothing (its da may be infinite)
  if (fa != 0.0f) r.z += fa * a.z, r.w += fa * (a.w + da * a.z);
  if (fb != 0.0f) r.z += fb * b.z, r.w += fb * (b.w + db * b.z);
  return r;
}
__device__ __forceinline__ Stats warp_merge(Stats a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = merge(a, Stats{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.z, o),
                       __shfl_xor_sync(0xffffffffu, a.w, o)}, c);
  return a;
}

// Values as unsigned numbers in their order (every NaN above everything, -0 as 0).
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
  return x != x ? 0xffffffffu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ Key order_key(float x, int i) {
  return ((Key)order_bits(x) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float bits_value(uint32_t u) {
  return u == 0xffffffffu ? NAN : __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// A lower bound of the k-th largest of the CTA's `mine` (as order bits): see above.  Two barriers.
__device__ __forceinline__ uint32_t kth_bound(uint32_t mine, int k, uint32_t* s_warp) {
  uint32_t top = 0;
  for (int i = 0; i < (k + kWarps - 1) / kWarps; ++i) {
    top = __reduce_max_sync(0xffffffffu, mine);
    // one holder of the maximum leaves
    const uint32_t who = __ballot_sync(0xffffffffu, mine == top);
    if ((threadIdx.x & 31) == __ffs(who) - 1) mine = 0;
  }
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = top;
  __syncthreads();
  uint32_t least = s_warp[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) least = min(least, s_warp[i]);
  __syncthreads();
  return least;
}

struct TopShared {
  Key buf[kBuffer];
  Key best[32];
  uint32_t warp[kWarps];
  int count;
};

// The best k of the buffered keys, in order, at the buffer's start; `count` becomes at most k.
// All threads; a key's rank is the number of larger ones.
__device__ __forceinline__ void compact(TopShared* s, int k) {
  __syncthreads();
  const int n = min(s->count, kBuffer);
  if (threadIdx.x < 32) s->best[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key mine = s->buf[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += s->buf[j] > mine;
    if (rank < k) s->best[rank] = mine;
  }
  __syncthreads();
  if (threadIdx.x < k) s->buf[threadIdx.x] = s->best[threadIdx.x];
  if (threadIdx.x == 0) s->count = min(n, k);
  __syncthreads();
}

// Offers the thread's keys (key_at(e), e < n <= 32) above *floor to the buffer; when it is full,
// the best k stay, the floor rises and what is left is offered again.  All threads.
template <int n, typename F>
__device__ __forceinline__ void offer(TopShared* s, int k, bool any, Key* floor, F key_at) {
  uint32_t left = any ? (n == 32 ? ~0u : (1u << n) - 1) : 0u;
  for (;;) {
    if (left) {
#pragma unroll
      for (int e = 0; e < n; ++e) {
        if (!(left >> e & 1)) continue;
        const Key key = key_at(e);
        if (key > *floor) {
          const int at = atomicAdd(&s->count, 1);
          if (at >= kBuffer) continue;                // stays on the list
          s->buf[at] = key;
        }
        left &= ~(1u << e);
      }
    }
    if (!__syncthreads_or(left != 0)) return;
    compact(s, k);
    *floor = s->buf[k - 1];                           // (it was full: there are k)
  }
}

struct Pieces {                            // how the line is cut
  long long granules;                      // of a row
  int ctas;                                // that have a part
  float c;                                 // scale log2 e
  float4* stats;                           // [row + cta]: m, z, w
  Key* keys;                               // [row + cta][k]
};

__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long p, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(*a), "=f"(*b) : "l"(p));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
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
__device__ __forceinline__ uint4 no_logits(const __nv_bfloat16*) {
  return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
}
__device__ __forceinline__ uint4 no_logits(const float*) {
  return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
}

// 16 bytes of logits from the 16-byte boundary at or below row + i on (i: the index of the first,
// which may lie before the row), -inf in the place of what is not the row's.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, long long i, int V) {
  constexpr int kVec = Granule<T>::kVec;
  if (i >= 0 && i + kVec <= V) {
    uint4 u;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(row + i));
    return u;
  }
  uint4 u = no_logits(row);
  if (i + kVec <= 0 || i >= V) return u;
  T* e = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int q = 0; q < kVec; ++q)
    if (i + q >= 0 && i + q < V) e[q] = row[i + q];
  return u;
}

template <typename T, bool kTop, bool kEntropy>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    gdn_token_logprobs_kernel(GdnLogprobArgs a, Pieces p) {
  using G = Granule<T>;
  __shared__ TopShared s_top;
  __shared__ Stats s_stats[kWarps];
  const int tid = threadIdx.x, cta = blockIdx.x;
  pdl_trigger();                                      // the joining kernel may be set up
  const long long total = p.granules * a.N;
  long long at = total * cta / p.ctas;
  const long long end = total * (cta + 1) / p.ctas;
  int row = (int)(at / p.granules);
  long long q = at - row * p.granules;                // granule of the row
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  // the row's first vector starts at its 16-byte boundary: `shift` logits before it
  auto shift_of = [&](const T* r) {
    return (int)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T));
  };
  int shift = shift_of(x);
  auto index = [&](long long g, int v) {
    return (g * 2 + v) * (long long)(kThreads * G::kVec) + tid * G::kVec - shift;
  };
  uint4 next[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) next[v] = load_vec(x, index(q, v), a.V);
  while (at < end) {
    // ---- this CTA's piece of a row: granules [q, q1)
    const long long left = end - at;
    const long long q1 = q + left < p.granules ? q + left : p.granules;
    float m = -INFINITY;
    unsigned long long z2 = 0, w2 = 0;                // pairs of sums
    bool nan = false;
    Key floor = 0;
    bool first = true;
    const unsigned long long c2 = pair(p.c, p.c);
    for (; q < q1; ++q, ++at) {
      uint4 now[2] = {next[0], next[1]};
      const long long i0 = index(q, 0), i1 = index(q, 1);
      // the granule after this one, of this row or the next
      if (at + 1 < end) {
        if (q + 1 == p.granules) {
          const T* nx = x + a.row_stride;
          const int keep = shift;
          shift = shift_of(nx);
#pragma unroll
          for (int v = 0; v < 2; ++v) next[v] = load_vec(nx, index(0, v), a.V);
          shift = keep;
        } else {
#pragma unroll
          for (int v = 0; v < 2; ++v) next[v] = load_vec(x, index(q + 1, v), a.V);
        }
      }
      float f[G::kPer];
      widen(now[0], x, f);
      widen(now[1], x, f + G::kVec);
      float top = f[0];
#pragma unroll
      for (int e = 1; e < G::kPer; ++e) top = max_nan(top, f[e]);
      nan = nan || top != top;
      if (top > m) {                                  // seldom after the first granules
        const float d = (m - top) * p.c, s = ptx::ex2_approx(d);
        const unsigned long long s2 = pair(s, s);
        if (s != 0.0f) {
          w2 = mul2(fma2(z2, pair(d, d), w2), s2);
          z2 = mul2(z2, s2);
        } else {
          w2 = z2 = 0;
        }
        m = top;
      }
      if (m != -INFINITY) {
        const unsigned long long minus_m = pair(-m, -m);
#pragma unroll
        for (int e = 0; e < G::kPer; e += 2) {
          float t0, t1;
          unpair(mul2(add2(pair(f[e], f[e + 1]), minus_m), c2), &t0, &t1);
          const unsigned long long e2 = pair(ptx::ex2_approx(t0), ptx::ex2_approx(t1));
          z2 = add2(z2, e2);
          // 0 * -inf is no part of the sum
          if (kEntropy) w2 = fma2(e2, pair(fmaxf(t0, -1000.0f), fmaxf(t1, -1000.0f)), w2);
        }
      }
      if constexpr (kTop) {
        if (first) {
          if (tid == 0) s_top.count = 0;
          const uint32_t bound = kth_bound(order_bits(top), a.top_k, s_top.warp);
          floor = bound ? ((Key)bound << 32) - 1 : 0;
          first = false;
        }
        auto key_at = [&](int e) {
          return order_key(f[e], (int)(e < G::kVec ? i0 + e : i1 + e - G::kVec));
        };
        // (index 0 ranks first among equal values)
        offer<G::kPer>(&s_top, a.top_k, order_key(top, 0) > floor, &floor, key_at);
      }
    }
    // ---- the piece's statistics and best k
    float z0, z1, w0, w1;
    unpair(z2, &z0, &z1);
    unpair(w2, &w0, &w1);
    Stats st{m, nan ? NAN : z0 + z1, w0 + w1};
    st = warp_merge(st, p.c);
    if ((tid & 31) == 0) s_stats[tid >> 5] = st;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int i = 1; i < kWarps; ++i) st = merge(st, s_stats[i], p.c);
      p.stats[(long long)row + cta] = make_float4(st.m, st.z, st.w, 0.0f);
    }
    if constexpr (kTop) {
      compact(&s_top, a.top_k);
      if (tid < a.top_k)
        p.keys[((long long)row + cta) * a.top_k + tid] = tid < s_top.count ? s_top.buf[tid] : 0;
    }
    __syncthreads();
    if (q == p.granules) {
      q = 0;
      ++row;
      x += a.row_stride;
      shift = shift_of(x);
    }
  }
}

// Joins a row's pieces: one CTA a row (a warp's worth without alternatives).
template <typename T, bool kTop>
__global__ void __launch_bounds__(kTop ? kThreads : 32)
    gdn_token_logprobs_join_kernel(GdnLogprobArgs a, Pieces p) {
  const int row = blockIdx.x, tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  const long long total = p.granules * a.N, x0 = row * p.granules, x1 = x0 + p.granules - 1;
  // the CTAs that hold the row's first and last granule
  const int c0 = (int)(((x0 + 1) * p.ctas - 1) / total), c1 = (int)(((x1 + 1) * p.ctas - 1) / total);
  pdl_wait();
  Stats st{-INFINITY, 0.0f, 0.0f};
  if (tid < 32) {
    for (int c = c0 + tid; c <= c1; c += 32) {
      const float4 v = p.stats[(long long)row + c];
      st = merge(st, Stats{v.x, v.y, v.z}, p.c);
    }
    st = warp_merge(st, p.c);
  }
  const bool dead = st.m == -INFINITY && st.z == 0.0f;  // every logit -inf
  const float log2z = log2f(st.z);
  auto logp = [&](float v) { return dead ? -INFINITY : (v - st.m) * a.scale - kLn2 * log2z; };
  if (tid == 0) {
    if (a.logprobs) {
      const int id = a.targets[row];
      float lp = 0.0f;
      if (id >= a.V) {
        atomicOr(&g_err_lp, kErrIndex);
        lp = NAN;
      } else if (id >= 0) {
        lp = logp(ld_elem(x + id));
      }
      a.logprobs[row] = lp;
    }
    if (a.entropy) a.entropy[row] = dead ? 0.0f : kLn2 * (log2z - st.w / st.z);
  }
  if constexpr (kTop) {
    __shared__ TopShared s_top;
    const int k = a.top_k;
    const long long n = (long long)(c1 - c0 + 1) * k;
    const Key* keys = p.keys + ((long long)row + c0) * k;   // the pieces' lists lie side by side
    Key best = 0;
    for (long long i = tid; i < n; i += kThreads) {
      const Key key = keys[i];
      best = key > best ? key : best;
    }
    if (tid == 0) s_top.count = 0;
    const uint32_t bound = kth_bound((uint32_t)(best >> 32), k, s_top.warp);
    Key floor = bound ? ((Key)bound << 32) - 1 : 0;
    for (long long i0 = 0; i0 < n; i0 += kThreads) {
      const Key key = i0 + tid < n ? keys[i0 + tid] : 0;
      offer<1>(&s_top, k, key > floor, &floor, [&](int) { return key; });
    }
    compact(&s_top, k);
    if (tid < k) {
      const Key key = s_top.buf[tid];
      const uint32_t bits = (uint32_t)(key >> 32);
      a.top_ids[(long long)row * k + tid] = (int)~(uint32_t)key;
      a.top_logprobs[(long long)row * k + tid] = logp(bits_value(bits));
    }
  }
}

template <typename T>
long long granules_of(int V) {             // with up to a vector's worth of shift
  return ((long long)V + Granule<T>::kVec - 1 + Granule<T>::kLogits - 1) / Granule<T>::kLogits;
}
long long granules_of(int V, int bf16) {
  return bf16 ? granules_of<__nv_bfloat16>(V) : granules_of<float>(V);
}
size_t stats_bytes(int N) { return (sizeof(float4) * ((size_t)N + kCtas) + 255) & ~(size_t)255; }

template <typename T, bool kTop, bool kEntropy>
cudaError_t launch(const GdnLogprobArgs& a, const Pieces& p, cudaStream_t stream) {
  gdn_token_logprobs_kernel<T, kTop, kEntropy><<<p.ctas, kThreads, 0, stream>>>(a, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(true, gdn_token_logprobs_join_kernel<T, kTop>, dim3((unsigned)a.N),
                    dim3(kTop ? kThreads : 32), 0, stream, a, p);
}

template <typename T>
cudaError_t launch(const GdnLogprobArgs& a, const Pieces& p, cudaStream_t stream) {
  if (a.top_k > 0)
    return a.entropy ? launch<T, true, true>(a, p, stream) : launch<T, true, false>(a, p, stream);
  return a.entropy ? launch<T, false, true>(a, p, stream) : launch<T, false, false>(a, p, stream);
}

}  // namespace

size_t gdn_token_logprobs_bytes(int N, int V, int bf16, int top_k) {
  (void)V;
  (void)bf16;
  return stats_bytes(N) + sizeof(Key) * top_k * ((size_t)N + kCtas);
}

cudaError_t gdn_launch_token_logprobs(const GdnLogprobArgs& a, cudaStream_t stream) {
  Pieces p;
  p.granules = granules_of(a.V, a.bf16);
  const long long total = p.granules * a.N;
  p.ctas = (int)(total < kCtas ? total : kCtas);
  p.c = a.scale * kLog2e;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.stats = reinterpret_cast<float4*>(ws);
  p.keys = reinterpret_cast<Key*>(ws + stats_bytes(a.N));
  return a.bf16 ? launch<__nv_bfloat16>(a, p, stream) : launch<float>(a, p, stream);
}
