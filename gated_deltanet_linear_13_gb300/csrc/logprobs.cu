// Log probabilities of given tokens with entropy and top alternatives, in one pass over the
// logits.
//
// Per set of logits x: the maximum m, z = sum 2^t and w = sum 2^t t with t = (x - m) scale log2 e;
// two sets join by rescaling to the larger maximum.  Then logp(i) = (x_i - m) scale - ln z and the
// entropy is ln 2 (log2 z - w / z): centred on m, so that nothing cancels and nothing overflows
// however large the logits are.  t is x c - m c in one rounding where m c is small enough for its
// own rounding to be made up for afterwards, and (x - m) c elsewhere.
//
// The alternatives cost the pass one maximum a granule (the kilobyte that a warp takes at a time).
// The k granules with the largest maxima hold the k best logits: a logit of another granule is
// beaten by the largest of each of the k.  (Granules are consecutive, so this holds for equal
// values too, which go by the lower index.)  The joining kernel finds the k-th largest of the
// row's maxima by counting, reads those granules again (k kilobytes of a row of hundreds), and
// gathers what reaches that maximum: vectors of 16 bytes, then their logits, a few more than k of
// them.  A logit's place is the number of better ones.  Where more pass than there is room for
// (rows of equal logits, rising rows) a warp keeps the best 32 vectors in order instead, one a
// lane, and the best 32 of their logits: a single better one is inserted (a ballot gives its
// place, a shuffle moves the rest up), many at once are sorted and merged.  A value and an index
// make one 64-bit key, ordered by value (NaN first, -0 equal to 0) and then by lower index; keys
// are distinct, so the result depends on no order of execution.
//
// All rows lie on one line of granules (the last of a row shorter), cut into equal parts, a warp's
// each, so that one long row fills the GPU as well as twenty thousand short ones; no warp waits for
// another.
//
// Bound by memory: each logit is read once.  At the copy rate an SM gets 12 bf16 logits a cycle,
// for which it can issue 128 lane operations; a logit takes about nine (packed fp32 pairs where
// there are such instructions) and one of 16 exponentials a cycle.  Measured: 1000 rows of 151669
// in fp32 101 us (6.0 TB/s); 64 rows of 248320 in bf16 with 20 alternatives 16.9 us, of which the
// pass takes 11 and the join 6; one row 8.8 us, two launches.
#include <float.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

using namespace gdn;
using ptx::add2;
using ptx::fma2;
using ptx::mul2;
using ptx::pair;
using ptx::unpair;

static __device__ unsigned int g_err_lp;

unsigned gdn_take_error_logprobs() { return gdn::take_error(g_err_lp); }

namespace {

typedef unsigned long long Key;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4, kParts = 152 * kCtasPerSm * kWarps;
// of a lane in the joining kernel: granules' maxima held, loads ahead of granules (two: 1400 rows
// of 32000 with 20 alternatives 44.6 us, four: 39.8, eight: 38.0, but 3000 rows 70.6 for 60.2) and
// of logits
constexpr int kHeld = 16, kGranulesAhead = 4, kLogitsAhead = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename T>
struct Granule {
  static constexpr int kVec = 16 / (int)sizeof(T);     // logits of a 16-byte vector
  static constexpr int kPer = 2 * kVec;                // of a lane
  static constexpr int kLogits = 32 * kPer;
};

// m = -inf: no logit above -inf.  A NaN among the logits: z is NaN.
struct Stats {
  float m, z, w;
};

__device__ __forceinline__ Stats merge(const Stats& a, const Stats& b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY || a.z != a.z || b.z != b.z) return Stats{m, a.z + b.z, a.w + b.w};
  const float da = scaled_difference(a.m, m, c), db = scaled_difference(b.m, m, c);
  const float fa = ptx::ex2_approx(da), fb = ptx::ex2_approx(db);
  Stats r{m, 0.0f, 0.0f};
  // a side that underflows adds nothing (its da may be infinite)
  if (fa != 0.0f) r.z += fa * a.z, r.w += fa * (a.w + da * a.z);
  if (fb != 0.0f) r.z += fb * b.z, r.w += fb * (b.w + db * b.z);
  return r;
}
__device__ __forceinline__ Stats other_lane(const Stats& a, int o) {
  return Stats{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.z, o),
               __shfl_xor_sync(0xffffffffu, a.w, o)};
}
__device__ __forceinline__ Stats warp_merge(Stats a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = merge(a, other_lane(a, o), c);
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

__device__ __forceinline__ Key key_max(Key a, Key b) { return a > b ? a : b; }
__device__ __forceinline__ Key key_min(Key a, Key b) { return a > b ? b : a; }

// The warp's best 32 keys so far, lane i the i-th (0: none); `floor` is the k-th, or a larger one
// that k keys of the row are known to reach.
struct Best {
  Key mine, floor;

  __device__ __forceinline__ void start() { mine = floor = 0; }
  __device__ __forceinline__ void set_floor(int k) {
    floor = key_max(floor, __shfl_sync(0xffffffffu, mine, k - 1));
  }
  __device__ __forceinline__ static Key exchange(Key x, int o, bool larger) {
    const Key y = __shfl_xor_sync(0xffffffffu, x, o);
    return larger ? key_max(x, y) : key_min(x, y);
  }
  // 32 keys, one a lane, into descending order (bitonic)
  __device__ __forceinline__ static Key sorted(Key x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
      for (int o = n >> 1; o > 0; o >>= 1)
        x = exchange(x, o, ((lane & o) == 0) == ((lane & n) == 0 || n == 32));
    return x;
  }
  // 32 keys in descending order join
  __device__ __forceinline__ void join(Key other, int k) {
    const int lane = threadIdx.x & 31;
    mine = key_max(mine, __shfl_sync(0xffffffffu, other, 31 - lane));   // the best 32, bitonic
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine = exchange(mine, o, (lane & o) == 0);
    set_floor(k);
  }
  // each lane's key, those above the floor join (all lanes)
  __device__ __forceinline__ void offer(Key key, int k) {
    uint32_t who = __ballot_sync(0xffffffffu, key > floor);
    if (who == 0) return;
    if (__popc(who) > 6) {                 // about what sorting and merging costs in insertions
      join(sorted(key > floor ? key : 0), k);
      return;
    }
    const int lane = threadIdx.x & 31;
    while (who) {
      const Key one = __shfl_sync(0xffffffffu, key, __ffs(who) - 1);
      who &= who - 1;
      const int place = __popc(__ballot_sync(0xffffffffu, mine > one));
      const Key up = __shfl_up_sync(0xffffffffu, mine, 1);
      mine = lane < place ? mine : lane == place ? one : up;
    }
    set_floor(k);
  }
  // N keys of each lane.  Without a floor, the lanes' largest come first (32 distinct keys): the
  // floor is then near its place, and few of the others pass it.
  template <int N>
  __device__ __forceinline__ void offer_all(Key (&key)[N], int k) {
    if (floor == 0 && __shfl_sync(0xffffffffu, mine, 0) == 0) {
      Key top = key[0];
#pragma unroll
      for (int i = 1; i < N; ++i) top = key_max(top, key[i]);
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = key[i] == top ? 0 : key[i];
      mine = sorted(top);
      set_floor(k);
    }
    uint32_t any = 0;                      // (one copy of the code for all N)
#pragma unroll
    for (int i = 0; i < N; ++i) any |= key[i] > floor ? 1u << i : 0u;
    any = __reduce_or_sync(0xffffffffu, any);
#pragma unroll 1
    while (any) {
      const int i = __ffs(any) - 1;
      any &= any - 1;
      Key one = key[0];
#pragma unroll
      for (int j = 1; j < N; ++j) one = i == j ? key[j] : one;
      offer(one, k);
    }
  }
};

struct Pieces {                            // how the line is cut
  long long total;                         // granules of all rows
  int granules;                            // of a row
  int parts;                               // equal parts of the line, a warp's each
  float c;                                 // scale log2 e
  float least;                             // logits above this stay finite when scaled by c
  float4* stats;                           // [row + part]: m, z, w
  uint32_t* tops;                          // [row][granule]: the largest logit's order bits
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
template <typename T>
__device__ __forceinline__ uint4 load_inner(const T* at) {
  uint4 u;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(at));
  return u;
}

// 16 bytes of logits from the 16-byte boundary at or below row + i on (i: the index of the first,
// which may lie before the row), -inf in the place of what is not the row's.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, long long i, int V) {
  constexpr int kVec = Granule<T>::kVec;
  if (i >= 0 && i + kVec <= V) return load_inner(row + i);
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

template <typename T, bool kTop, bool kEntropy>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    gdn_token_logprobs_kernel(GdnLogprobArgs a, Pieces p) {
  using G = Granule<T>;
  constexpr int kDepth = 2;                           // granules on the way
  const int lane = threadIdx.x & 31, part = blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_trigger();                                      // the joining kernel may be set up
  if (part >= p.parts) return;
  const long long start = p.total * part / p.parts;
  int left = (int)(p.total * (part + 1) / p.parts - start);
  int row = (int)(start / p.granules);
  int q = (int)(start - (long long)row * p.granules); // granule of the row
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  // the granules ahead: (row, granule) of the next to be loaded and this lane's place in it
  const T* ax = x;
  int aq = q, aleft = left;
  const T* ap = ax - shift_of(ax) + (long long)aq * G::kLogits + lane * G::kVec;
  uint4 ahead[kDepth][2];
  auto load = [&](uint4 (&to)[2]) {
    if (aleft <= 0) return;
    if (aq > 0 && aq + 2 < p.granules) {              // all of it the row's
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const T* at = ap + v * 32 * G::kVec;
        if (in_bounds(&g_err_lp, at >= ax && at + G::kVec <= ax + a.V)) to[v] = load_inner(at);
      }
    } else {
#pragma unroll
      for (int v = 0; v < 2; ++v) to[v] = load_vec(ax, ap - ax + v * 32 * G::kVec, a.V);
    }
    --aleft;
    ap += G::kLogits;
    if (++aq == p.granules) {
      aq = 0;
      ax += a.row_stride;
      ap = ax - shift_of(ax) + lane * G::kVec;
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(ahead[i]);
  const unsigned long long c2 = pair(p.c, p.c);
  while (left > 0) {
    // ---- this warp's granules of a row
    float m = -INFINITY, above = INFINITY;            // (see below)
    unsigned long long z2 = 0, w2 = 0;                // pairs of sums
    const int q0 = q, q1 = q + left < p.granules ? q + left : p.granules;
#pragma unroll kDepth
    for (; q < q1; ++q) {
      float f[G::kPer], top, least;
      widen(ahead[0][0], x, f);
      widen(ahead[0][1], x, f + G::kVec);
      range(ahead[0][0], ahead[0][1], x, f, &top, &least);
#pragma unroll
      for (int i = 0; i + 1 < kDepth; ++i) {
        ahead[i][0] = ahead[i + 1][0];
        ahead[i][1] = ahead[i + 1][1];
      }
      load(ahead[kDepth - 1]);
      if (top > m) {                                  // seldom after the first granules
        // The sums' reference is m c as it rounds where that is near, else m c itself.  They go
        // from one to the next by both roundings, or what is summed so far loses its weight.
        const float d = reference_difference(m, top, p.c);
        const float s = ptx::ex2_approx(d);
        const unsigned long long s2 = pair(s, s);
        w2 = s != 0.0f ? mul2(fma2(z2, pair(d, d), w2), s2) : 0;
        z2 = mul2(z2, s2);                            // (a NaN stays)
        m = top;
        above = fabsf(m * p.c) <= kNear ? p.least : INFINITY;
      }
      const float mc = m * p.c;
      if (least > above) {
        // t = x c - mc in one rounding; that mc is rounded the sums make up for at the end
        const unsigned long long minus_mc = pair(-mc, -mc);
#pragma unroll
        for (int e = 0; e < G::kPer; e += 2) {
          const unsigned long long t2 = fma2(pair(f[e], f[e + 1]), c2, minus_mc);
          float t0, t1;
          unpair(t2, &t0, &t1);
          const unsigned long long e2 = pair(ptx::ex2_approx(t0), ptx::ex2_approx(t1));
          z2 = add2(z2, e2);
          if (kEntropy) w2 = fma2(e2, t2, w2);
        }
      } else if (m != -INFINITY || top != top) {
        // infinite logits among them, or a reference too large to be taken off after scaling:
        // then t = (x - m) c
        const bool near = fabsf(mc) <= kNear;
        const float sub = near ? 0.0f : m, base = near ? mc : 0.0f;
        const unsigned long long minus_sub = pair(-sub, -sub), minus_base = pair(-base, -base);
#pragma unroll
        for (int e = 0; e < G::kPer; e += 2) {
          float t0, t1;
          unpair(fma2(add2(pair(f[e], f[e + 1]), minus_sub), c2, minus_base), &t0, &t1);
          const unsigned long long e2 = pair(ptx::ex2_approx(t0), ptx::ex2_approx(t1));
          z2 = add2(z2, e2);
          // 0 * -inf is no part of the sum
          w2 = fma2(e2, pair(fmaxf(t0, -1000.0f), fmaxf(t1, -1000.0f)), w2);
        }
      }
      if constexpr (kTop) {
        const uint32_t bits = __reduce_max_sync(0xffffffffu, order_bits(top));
        if (lane == 0 && in_bounds(&g_err_lp, row < a.N && q < p.granules))
          p.tops[(long long)row * p.granules + q] = bits;
      }
    }
    left -= q1 - q0;
    // ---- their statistics
    float z0, z1, w0, w1;
    unpair(z2, &z0, &z1);
    unpair(w2, &w0, &w1);
    const float z = z0 + z1, off = rounding(m, p.c), up = ptx::ex2_approx(-off);
    const Stats st = warp_merge(Stats{m, z * up, (w0 + w1 - off * z) * up}, p.c);
    if (lane == 0 && in_bounds(&g_err_lp, row < a.N && part < kParts))
      p.stats[(long long)row + part] = make_float4(st.m, st.z, st.w, 0.0f);
    if (q == p.granules) {
      q = 0;
      ++row;
      x += a.row_stride;
    }
  }
}

// The best k of a row's granules by their largest logit, equal ones by the lower index, in
// ascending order into list; returns order bits that each of them reaches.  The k-th largest is
// found bit by bit, counting what reaches a number (a warp's sum is one instruction), and as soon
// as exactly k do, those are the ones.  A bf16 number's order bits differ in the upper half only.
template <typename T>
__device__ __forceinline__ uint32_t best_granules(const uint32_t* tops, int granules, int k,
                                                  const uint32_t (&held)[kHeld], int* list) {
  constexpr int kLow = sizeof(T) == 2 ? 16 : 0;
  const int lane = threadIdx.x & 31;
  auto each = [&](auto&& f) {              // the row's maxima, 32 at a time; 0 past the end
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i * 32 < granules) f(i * 32 + lane, held[i]);
#pragma unroll 4
    for (int q = kHeld * 32 + lane; q - lane < granules; q += 32)
      f(q, q < granules ? tops[q] : 0u);
  };
  uint32_t most = 0, least = 0xffffffffu;
  each([&](int q, uint32_t v) {
    most = max(most, v);
    if (q < granules) least = min(least, v);
  });
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  auto reach = [&](uint32_t y) {
    int n = 0;
    each([&](int, uint32_t v) { n += v >= y ? 1 : 0; });
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  };
  // their common leading bits, then the others
  uint32_t x = most;
  int b = 31 - __clz(most ^ least);
  if (b >= kLow) x &= ~((2u << b) - 1u);
#pragma unroll 1
  for (; b >= kLow; --b) {
    const uint32_t y = x | 1u << b;
    const int n = reach(y);
    if (n >= k) x = y;
    if (n == k) break;
  }
  x &= ~((1u << kLow) - 1u);
  const uint32_t over = x + (1u << kLow);  // (0: nothing is)
  int ties = k - (over ? reach(over) : 0), taken = 0;
  const uint32_t before = (1u << lane) - 1u;
  each([&](int q, uint32_t v) {
    if (taken >= k) return;
    const bool more = over && v >= over, tie = v >= x && !more;
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    const bool take = more || (tie && __popc(tied & before) < ties);
    const uint32_t took = __ballot_sync(0xffffffffu, take);
    if (take) list[taken + __popc(took & before)] = q;
    ties -= min(ties, __popc(tied));
    taken += __popc(took);
  });
  return x;
}

// Joins a row's pieces: kRowWarps warps a row (1: a few pieces; 8: many, which the warps share).
template <typename T, bool kTop, int kRowWarps>
__global__ void __launch_bounds__(kThreads)
    gdn_token_logprobs_join_kernel(GdnLogprobArgs a, Pieces p) {
  constexpr int kVec = Granule<T>::kVec;
  // a row's candidates: vectors, then logits
  constexpr int kVectors = kTop ? 64 : 1, kMost = kTop ? 64 : 1;
  constexpr int kSlots = kTop ? kWarps / kRowWarps : 1;               // rows of a block
  __shared__ Stats s_stats[kWarps];
  __shared__ Key s_best[kTop ? kWarps : 1][32];
  __shared__ uint4 s_vector[kSlots][kVectors];
  __shared__ int s_index[kSlots][kVectors];
  __shared__ __align__(16) Key s_candidate[kSlots][kMost];
  __shared__ int s_granule[kSlots][32];
  __shared__ uint32_t s_floor[kSlots];
  __shared__ int s_vectors[kSlots], s_candidates[kSlots];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = kRowWarps == 1 ? 0 : warp, slot = kRowWarps == 1 ? warp : 0;
  const long long row = kRowWarps == 1 ? (long long)blockIdx.x * kWarps + warp : blockIdx.x;
  if (row >= a.N) return;                             // (whole blocks where warps share a row)
  auto sync = [&]() {                                 // the row's warps
    if constexpr (kRowWarps == 1) __syncwarp();
    else __syncthreads();
  };
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  const long long x0 = row * p.granules, x1 = x0 + p.granules - 1;
  // the parts that hold the row's first and last granule
  const int c0 = (int)(((x0 + 1) * p.parts - 1) / p.total);
  const int pieces = (int)(((x1 + 1) * p.parts - 1) / p.total) - c0 + 1;
  const int id = a.logprobs && sub == 0 ? a.targets[row] : -1;
  const float target = id >= 0 && id < a.V ? ld_elem(x + id) : 0.0f;
  if (kTop && lane == 0 && sub == 0) s_vectors[slot] = s_candidates[slot] = 0;
  pdl_wait();
  const int shift = shift_of(x), n = min(a.top_k, p.granules);
  int granule = lane;                                 // lane i the i-th of the best (or of all)
  uint32_t floor = 0;                                 // k logits reach it
  // the first warp finds the granules, the others join the statistics
  const bool selects = kTop && sub == 0 && p.granules > a.top_k;
  if constexpr (kTop) {
    if (selects) {
      const uint32_t* tops = p.tops + row * p.granules;
      uint32_t held[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int q = i * 32 + lane;
        held[i] = q < p.granules ? tops[q] : 0u;
      }
      floor = best_granules<T>(tops, p.granules, a.top_k, held, s_granule[slot]);
      if (lane == 0) s_floor[slot] = floor;
    }
  }
  Stats st{-INFINITY, 0.0f, 0.0f};
  constexpr int kOthers = kTop && kRowWarps > 1 ? kRowWarps - 1 : kRowWarps;
  for (int i = (sub - (kRowWarps - kOthers)) * 32 + lane; i >= 0 && i < pieces; i += kOthers * 32) {
    if (!in_bounds(&g_err_lp, c0 >= 0 && c0 + i < kParts)) break;
    const float4 v = p.stats[row + c0 + i];
    st = merge(st, Stats{v.x, v.y, v.z}, p.c);
  }
  if (kRowWarps == 1 || kOthers == kRowWarps || sub > 0) st = warp_merge(st, p.c);
  if (kRowWarps > 1 && lane == 0) s_stats[warp] = st;
  if constexpr (kTop) {
    sync();
    if (p.granules > a.top_k) granule = s_granule[slot][lane], floor = s_floor[slot];
    if (lane < n && !in_bounds(&g_err_lp, granule >= 0 && granule < p.granules)) granule = 0;
    // their vectors that reach it
    for (int i0 = sub; i0 < n; i0 += kRowWarps * kGranulesAhead) {
      uint4 u[2 * kGranulesAhead];
      int vec[2 * kGranulesAhead];
#pragma unroll
      for (int i = 0; i < kGranulesAhead; ++i) {
        const int at = i0 + i * kRowWarps, q = __shfl_sync(0xffffffffu, granule, at & 31);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          vec[2 * i + v] = at < n ? q * 64 + v * 32 + lane : -1;
          u[2 * i + v] = at < n ? load_vec(x, (long long)vec[2 * i + v] * kVec - shift, a.V)
                                : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < 2 * kGranulesAhead; ++j) {
        if (vec[j] < 0 || order_bits(vector_top(u[j], x)) < floor) continue;
        const int to = atomicAdd(&s_vectors[slot], 1);
        if (to >= kVectors) continue;
        s_vector[slot][to] = u[j];
        s_index[slot][to] = vec[j];
      }
    }
    sync();
    // and those vectors' logits
    const int logits = min(s_vectors[slot], kVectors) * kVec;
    for (int i = sub * 32 + lane; i < logits; i += kRowWarps * 32) {
      const int e = i % kVec;
      const T* words = reinterpret_cast<const T*>(&s_vector[slot][i / kVec]);
      const float f = ld_elem(words + e);
      const long long at = (long long)s_index[slot][i / kVec] * kVec + e - shift;
      if (order_bits(f) < floor || at < 0 || at >= a.V) continue;
      const int to = atomicAdd(&s_candidates[slot], 1);
      if (to < kMost) s_candidate[slot][to] = order_key(f, (int)at);
    }
  }
  if (kTop || kRowWarps > 1) sync();
  if constexpr (kRowWarps > 1) {
    st = s_stats[lane & (kWarps - 1)];                // every eight lanes hold all of them
    for (int o = kWarps / 2; o > 0; o >>= 1) st = merge(st, other_lane(st, o), p.c);
  }
  const bool dead = st.m == -INFINITY && st.z == 0.0f;  // every logit -inf
  // (a merge rounds its two sides differently, so lanes may differ in the last bit)
  const float log2z = __shfl_sync(0xffffffffu, log2f(st.z), 0);
  auto logp = [&](float v) {
    return dead ? -INFINITY : scaled_difference(v, st.m, a.scale) - kLn2 * log2z;
  };
  auto store_top = [&](int rank, Key key) {
    if (!in_bounds(&g_err_lp, rank >= 0 && rank < a.top_k && ~(uint32_t)key < (uint32_t)a.V)) return;
    a.top_ids[row * a.top_k + rank] = (int)~(uint32_t)key;
    a.top_logprobs[row * a.top_k + rank] = logp(bits_value((uint32_t)(key >> 32)));
  };
  if (lane == 0 && sub == 0) {
    if (a.logprobs) {
      if (id >= a.V) atomicOr(&g_err_lp, kErrIndex);
      a.logprobs[row] = id >= a.V ? NAN : id >= 0 ? logp(target) : 0.0f;
    }
    if (a.entropy) a.entropy[row] = dead ? 0.0f : kLn2 * (log2z - st.w / st.z);
  }
  if constexpr (kTop) {
    const int candidates = s_candidates[slot];
    if (s_vectors[slot] <= kVectors && candidates <= kMost) {
      // a candidate's place: how many are better
      for (int i = sub * 32 + lane; i < candidates; i += kRowWarps * 32) {
        const Key key = s_candidate[slot][i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < candidates; ++j) rank += s_candidate[slot][j] > key ? 1 : 0;
        if (rank < a.top_k) store_top(rank, key);
      }
      return;
    }
    // Too many (equal logits, or rising ones): of each warp's granules the vectors that may be
    // among the best k, then the best k of those vectors' logits.
    Best best;
    best.start();
    if (floor != 0) best.floor = ((Key)floor << 32) - 1;
    for (int i0 = sub; i0 < n; i0 += kRowWarps * kGranulesAhead) {
      Key key[2 * kGranulesAhead];
#pragma unroll
      for (int i = 0; i < kGranulesAhead; ++i) {
        const int at = i0 + i * kRowWarps, q = __shfl_sync(0xffffffffu, granule, at & 31);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int vec = q * 64 + v * 32 + lane;
          const uint4 u = at < n ? load_vec(x, (long long)vec * kVec - shift, a.V)
                                 : make_uint4(0, 0, 0, 0);
          key[2 * i + v] = at < n ? order_key(vector_top(u, x), vec) : 0;
        }
      }
      best.offer_all(key, a.top_k);
    }
    if constexpr (kRowWarps > 1) {
      s_best[warp][lane] = best.mine;
      __syncthreads();
      if (warp > 0) return;
      // the lists' first four at once, then what else of them is good enough
      best.start();
      best.mine = Best::sorted(s_best[lane & (kWarps - 1)][lane / kWarps]);
      best.set_floor(a.top_k);
      for (int i = 0; i < kWarps; ++i) {
        const Key rest = lane >= 32 / kWarps ? s_best[i][lane] : 0;
        if (__any_sync(0xffffffffu, rest > best.floor)) best.offer(rest, a.top_k);
      }
    }
    // the logits of the best k vectors, a lane one at a time
    const int logits = a.top_k * kVec;
    const Key vector = best.mine;
    best.start();
    for (int i0 = 0; i0 < logits; i0 += 32 * kLogitsAhead) {
      Key key[kLogitsAhead];
#pragma unroll
      for (int j = 0; j < kLogitsAhead; ++j) {
        const int i = i0 + j * 32 + lane;
        const Key v = __shfl_sync(0xffffffffu, vector, (i / kVec) & 31);
        const long long at = (long long)(uint32_t)~(uint32_t)v * kVec + i % kVec - shift;
        key[j] = i < logits && v != 0 && at >= 0 && at < a.V ? order_key(ld_elem(x + at), (int)at)
                                                             : 0;
      }
      best.offer_all(key, a.top_k);
    }
    if (lane < a.top_k) store_top(lane, best.mine);
  }
}

int granules_of(int V, int bf16) {         // with up to a vector's worth of shift
  const int vec = bf16 ? Granule<__nv_bfloat16>::kVec : Granule<float>::kVec;
  const int per = bf16 ? Granule<__nv_bfloat16>::kLogits : Granule<float>::kLogits;
  return (int)(((long long)V + vec - 1 + per - 1) / per);
}

size_t stats_bytes(int N) {
  return (sizeof(float4) * ((size_t)N + kParts) + 255) & ~(size_t)255;
}

template <typename T, bool kTop, bool kEntropy>
cudaError_t launch(const GdnLogprobArgs& a, const Pieces& p, cudaStream_t stream) {
  const int grid = (p.parts + kWarps - 1) / kWarps;
  gdn_token_logprobs_kernel<T, kTop, kEntropy><<<grid, kThreads, 0, stream>>>(a, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Few rows: a CTA's warps share one.  With eight warps a row and with one, rows of 32000 bf16
  // logits: 20 alternatives, 300 rows 14.9 / 25.3 us, 1200 33.2 / 36.8, 1400 40.6 / 39.4; one, 300 rows
  // 13.7 / 15.8, 800 25.0 / 22.4 (fp32 31.8 / 32.3).  Without alternatives a row's few pieces are
  // all there is to join: 64 rows 6.1 / 6.3, 300 10.2 / 9.6, 1200 20.7 / 19.7; 8 rows of 248320 6.4 / 10.7.
  if (a.N <= (kTop ? 152 * 8 : 152))
    return launch_pdl(true, gdn_token_logprobs_join_kernel<T, kTop, kWarps>, dim3((unsigned)a.N),
                      dim3(kThreads), 0, stream, a, p);
  return launch_pdl(true, gdn_token_logprobs_join_kernel<T, kTop, 1>,
                    dim3((unsigned)((a.N + kWarps - 1ll) / kWarps)), dim3(kThreads), 0, stream, a, p);
}

template <typename T>
cudaError_t launch(const GdnLogprobArgs& a, const Pieces& p, cudaStream_t stream) {
  if (a.top_k > 0)
    return a.entropy ? launch<T, true, true>(a, p, stream) : launch<T, true, false>(a, p, stream);
  return a.entropy ? launch<T, false, true>(a, p, stream) : launch<T, false, false>(a, p, stream);
}

}  // namespace

size_t gdn_token_logprobs_bytes(int N, int V, int bf16, int top_k) {
  return stats_bytes(N) + (top_k ? sizeof(uint32_t) * (size_t)N * granules_of(V, bf16) : 0);
}

cudaError_t gdn_launch_token_logprobs(const GdnLogprobArgs& a, cudaStream_t stream) {
  Pieces p;
  p.granules = granules_of(a.V, a.bf16);
  p.total = (long long)p.granules * a.N;
  p.parts = (int)(p.total < kParts ? p.total : kParts);
  // twice it is finite too (a scale past 1e38 is cut short: differences below 1e-36 could tell)
  p.c = fminf(a.scale * kLog2e, 0.5f * FLT_MAX);
  p.least = -1e30f / p.c;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.stats = reinterpret_cast<float4*>(ws);
  p.tops = reinterpret_cast<uint32_t*>(ws + stats_bytes(a.N));
  return a.bf16 ? launch<__nv_bfloat16>(a, p, stream) : launch<float>(a, p, stream);
}
