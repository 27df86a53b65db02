// Verification of drafted tokens from given random numbers, and the draw of the token behind the
// last accepted one.
//
// With p = softmax(s x), q = softmax(s y) (x the target's logits, y the draft's): draft t is accepted
// while u_t < p(t) / q(t); behind the last accepted one the token is the first of exponential clocks
// E_i with rates w_i, argmax w_i / E_i, w = max(p - q, 0) after a refusal (which makes the tokens the
// target's own), w = p after the last draft.
//
// Two passes.  The first reads every row once: its largest logit m and z = sum e^(s (x - m)), as
// the token log probabilities do it, on one line of granules cut into equal parts (a warp's each).
// The second knows each sequence's accepted count from them, and runs the race over the one row
// pair that matters, the last sequences first, whose rows L2 still holds: a CTA a slice, the last
// CTA of a sequence joins the slices.  p's normaliser cancels in the race (w = e^.. - e^.. z_p / z_q),
// so without drafts the first pass runs it as it goes and the second only joins.
// A warp keeps the best w / E of its elements so far; an element is looked at closer only if
// w > best E, nearly, so there is a division where the best changes and none elsewhere.  Where two
// lanes' or slices' best are within 2^-16 of each other they are compared in 64 bits, and so is a u near
// its border.  m, z and a lane's own weights are in 32 bits: p and q are right to 2^-20 or so of
// themselves, and after a refusal p - q to that of p + q, however small it is.
//
// Bound by memory where the batch is large: 64 sequences of 4 drafts over 248320 logits in bf16 66 us
// (240 MB of rows in 42 us, 5.7 TB/s, then 90 MB), 128 draws of 151936 23 us (95 MB); by instructions
// and exponentials next to it (a granule of a row 130 instructions a warp, sixteen exponentials a
// lane).  By latency where it is small: one sequence of 3 drafts 11 us, of which the rows take 3.3,
// the second kernel's start behind the first 1.8, statistics and decisions 1.3, a slice 1.8, the join
// of the slices and the tokens 2.5.
// Part of logprobs.cu, whose error word it uses.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "logits.cuh"
#include "sm100_ptx.cuh"

using namespace gdn;
using ptx::add2;
using ptx::fma2;
using ptx::mul2;
using ptx::pair;
using ptx::unpair;

namespace {
namespace verify {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtasPerSm = 3, kRaceCtasPerSm = 3;
// of the pass that also draws: 128 rows of 151936 in bf16 24 us (three: registers spill, 39); 64 of 151936
// in fp32 18.5 us with two, 17.0 with three
constexpr int draw_ctas(bool bf16) { return bf16 ? 2 : 3; }
constexpr int kMaxRows = 2 * kGdnMaxDrafts + 1;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMost = 18446744073709551616.0f;       // 2^64: scales lie within it and its inverse
constexpr float kClose = 1.0f - 0x1p-16f;
// A tinier clock rings as this one, so that w / E stays finite: an infinite one is above larger ones, and
// is a NaN once its reference has moved far.
constexpr float kLeastClock = 0x1p-126f;

struct Plan {
  int granules;                            // of a row
  int rows;                                // of a sequence: T + 1 of the target, then the draft's
  int parts;                               // of the line of all rows' granules, a warp's each
  int each, more;                          // granules of a part, and the first `more` have one more
  int pieces;                              // slices of a sequence's race
  int slice;                               // logits of a slice
  long long room;                          // slices that the workspace holds, of all sequences
  float4* stats;                           // [row + part]: m, z, granule of the largest; where
                                           // the first pass draws: m, z, index (greedy:
                                           // granule), w / E
  float4* best;                            // [B][pieces]: w / E, its index and its logit
  int* done;                               // [B] (neither is there without drafts)
};

// A row's largest logit (m = -inf: none above it), z, and the first granule that holds it.
struct Row {
  float m, z;
  int q;
};

__device__ __forceinline__ Row merge(const Row& a, const Row& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const int q = a.m == b.m ? min(a.q, b.q) : a.m > b.m ? a.q : b.q;
  if (m == -INFINITY || a.z != a.z || b.z != b.z) return Row{m, a.z + b.z, q};
  // (where one is -inf its z is 0)
  const float za = a.m == -INFINITY ? 0.0f : a.z * ptx::ex2_approx((a.m - m) * c);
  const float zb = b.m == -INFINITY ? 0.0f : b.z * ptx::ex2_approx((b.m - m) * c);
  return Row{m, za + zb, q};
}
// A float's bits in the order of the numbers, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}
// The largest of the warp's (no NaN).
__device__ __forceinline__ float warp_max(float x) {
  return unordered(__reduce_max_sync(0xffffffffu, ordered(x)));
}
__device__ __forceinline__ Row warp_merge(const Row& a, float c) {
  const float m = warp_max(a.m);
  const int q = (int)__reduce_min_sync(0xffffffffu, a.m == m ? (unsigned)a.q : 0x7fffffffu);
  // (where m is -inf every z is 0 or NaN)
  const float z = a.m == m ? a.z : a.z * ptx::ex2_approx((a.m - m) * c);
  return Row{m, warp_sum(z), q};
}

// The sums' reference: a term is 2^(x c - base), base = m c as it rounds, in one rounding, where that
// is near enough; else 2^((x - m) c).  The first carry 2^rounding(m, c), which settled() takes out.
struct Reference {
  float m, base;
  bool near;

  __device__ __forceinline__ void start() { m = base = -INFINITY, near = false; }
  // moves to a larger m; returns what sums under the old one are multiplied by
  __device__ __forceinline__ float raise(float to, float c) {
    const float f = ptx::ex2_approx(reference_difference(m, to, c));   // (0 from -inf)
    m = to;
    base = to * c;
    near = fabsf(base) <= kNear;
    return f;
  }
  __device__ __forceinline__ float settled(float c) const { return ptx::ex2_approx(-rounding(m, c)); }
  // the terms of N numbers, two at a time to f
  template <int N, typename F>
  __device__ __forceinline__ void terms(const float (&x)[N], float c, F&& f) const {
    const unsigned long long c2 = pair(c, c);
    if (near) {
      const unsigned long long minus = pair(-base, -base);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        float t0, t1;
        unpair(fma2(pair(x[k], x[k + 1]), c2, minus), &t0, &t1);
        f(k, ptx::ex2_approx(t0), ptx::ex2_approx(t1));
      }
    } else {
      const unsigned long long minus = pair(-m, -m);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        float t0, t1;
        unpair(mul2(add2(pair(x[k], x[k + 1]), minus), c2), &t0, &t1);
        f(k, ptx::ex2_approx(t0), ptx::ex2_approx(t1));
      }
    }
  }
};

// load_vec with the vectors that are only partly the row's out of line (a call waits for its loads;
// in line they cost the loops registers).
template <typename T>
__device__ __noinline__ uint4 partial_vec(const T* row, long long i, int V) {
  return load_vec<false>(row, i, V);
}
template <bool kOnce, typename T>
__device__ __forceinline__ uint4 edge_vec(const T* row, long long i, int V) {
  constexpr int kVec = Granule<T>::kVec;
  constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;     // -inf
  uint4 u = make_uint4(kNone, kNone, kNone, kNone);
  if (i >= 0 && i + kVec <= V) u = load_inner<kOnce>(row + i);
  else if (i + kVec > 0 && i < V) u = partial_vec(row, i, V);
  return u;
}

// Granules [first, first + count) of the line.
struct Part {
  int first, count;
};
__device__ __forceinline__ Part part_at(const Plan& p, int part) {
  return Part{part * p.each + min(part, p.more), p.each + (part < p.more ? 1 : 0)};
}
// The part that granule x is in.
__device__ __forceinline__ int part_of(const Plan& p, int x) {
  const int wide = p.more * (p.each + 1);
  return x < wide ? (int)((unsigned)x / (unsigned)(p.each + 1))
                  : p.more + (int)((unsigned)(x - wide) / (unsigned)p.each);
}

__device__ __forceinline__ bool in_range(float s) { return s >= 1.0f / kMost && s <= kMost; }
__device__ __forceinline__ bool takes_part(float s) { return s == INFINITY || in_range(s); }
// a greedy sequence's probabilities are those of scale 1
__device__ __forceinline__ float scale_of(float s) { return s == INFINITY ? 1.0f : s; }

template <typename T>
__device__ __forceinline__ const T* row_at(const GdnVerifyArgs& a, int b, int j) {
  return j <= a.T ? static_cast<const T*>(a.target) + ((long long)b * (a.T + 1) + j) * a.target_stride
                  : static_cast<const T*>(a.draft) + ((long long)b * a.T + j - a.T - 1) * a.draft_stride;
}

// Drafts of sequence b: up to the first id that is none (the whole warp).
__device__ __forceinline__ int drafts_of(const GdnVerifyArgs& a, int b) {
  int n = 0;
  for (int t0 = 0; t0 < a.T; t0 += 32) {
    const int t = t0 + (threadIdx.x & 31);
    const int id = t < a.T ? a.ids[(long long)b * a.T + t] : -1;
    const uint32_t bad = __ballot_sync(0xffffffffu, (unsigned)id >= (unsigned)a.V);
    if (bad) return n + __ffs(bad) - 1;
    n += 32;
  }
  return n;
}

// w / E of element i in 64 bits (seldom: out of line, so that it costs the loops no registers).
template <typename T>
__device__ __noinline__ double exact_race(const T* x, const T* y, const float* clocks, float mx,
                                          float my, float ratio, float scale, int i) {
  double w = exp(((double)ld_elem(x + i) - (double)mx) * (double)scale);
  if (y) w -= exp(((double)ld_elem(y + i) - (double)my) * (double)scale) * (double)ratio;
  return w / (double)fmaxf(clocks[i], kLeastClock);
}

// (x - mx) - (y - my), finite and of any size, as if rounded once: where x and y are alike far below
// (masks of the type's lowest value) it is my - mx that is left (seldom, so out of line).
__device__ __noinline__ double difference_of(double x, double mx, double y, double my) {
  auto sum = [](double a, double b, double* lost) {
    const double s = a + b, t = s - a;
    *lost += (a - (s - t)) + (b - t);
    return s;
  };
  double lost = 0.0;
  const double xy = sum(x, -y, &lost), m = sum(my, -mx, &lost), all = sum(xy, m, &lost);
  return all + lost;
}

// The race of one row pair, as a warp runs it: the same best in all lanes.
template <typename T>
struct Race {
  const T* x;                              // the target's row
  const T* y;                              // the draft's, or NULL
  const float* clocks;
  float mx, my, c, ratio;                  // ratio: z_p / z_q
  float scale;
  int never;                               // the refused draft where q is all on it, or -1
  float best;                              // w / E
  int at;

  __device__ __forceinline__ void challenge(float r, int i) {
    bool wins = best == 0.0f || r * kClose > best;
    if (!wins && r >= best * kClose) {
      const double mine = exact_race(x, y, clocks, mx, my, ratio, scale, at);
      const double other = exact_race(x, y, clocks, mx, my, ratio, scale, i);
      wins = other > mine || (other == mine && i < at);
    }
    if (wins) best = r, at = i;
  }
  // the lanes' best (r = 0: none), one a lane
  __device__ __forceinline__ void join(float r, int i) {
    const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(r)));
    uint32_t who = __ballot_sync(0xffffffffu, r > 0.0f && r >= top * kClose);
    while (who) {                          // seldom more than one
      const int from = __ffs(who) - 1;
      who &= who - 1;
      challenge(__shfl_sync(0xffffffffu, r, from), __shfl_sync(0xffffffffu, i, from));
    }
  }
  // N elements of each lane, the k-th of index at(k)
  template <int N, typename At>
  __device__ __forceinline__ void offer(const float (&w)[N], const float (&e)[N], At&& at_of) {
    const float floor = best * kClose;
    float over = 0.0f;                     // (a NaN or an infinite clock stays below, a tiny one above)
    if constexpr (N % 2 == 0) {
      const unsigned long long minus = pair(-floor, -floor);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        float o0, o1;
        unpair(fma2(pair(e[k], e[k + 1]), minus, pair(w[k], w[k + 1])), &o0, &o1);
        over = fmaxf(over, fmaxf(o0, o1));
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) over = fmaxf(over, fmaf(-floor, e[k], w[k]));
    }
    if (!__any_sync(0xffffffffu, over > 0.0f)) return;
    float r = 0.0f;
    int at_k = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float clock = fmaxf(e[k], kLeastClock);
      if (!(e[k] > 0.0f && w[k] > 0.0f && w[k] > floor * clock && at_of(k) != never)) continue;
      const float q = __fdiv_rn(w[k], clock);
      if (q > r) r = q, at_k = at_of(k);
    }
    if (__any_sync(0xffffffffu, r > 0.0f)) join(r, at_k);
  }
};

// Whether row j of sequence b is needed: its drafts', and the one behind them (the whole warp).
__device__ __forceinline__ bool needed(const GdnVerifyArgs& a, int b, int j) {
  const int n = drafts_of(a, b);
  return takes_part(a.scale ? a.scale[b] : 1.0f) && (j <= a.T ? j <= n : j - a.T - 1 < n);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) gdn_verify_rows_kernel(GdnVerifyArgs a,
                                                                              Plan p) {
  using G = Granule<T>;
  constexpr int kDepth = 2;                // granules on the way
  const int lane = threadIdx.x & 31, part = blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_wait();                              // (nothing is read before)
  pdl_trigger();
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.B; b += gridDim.x * kThreads) p.done[b] = 0;
  if (part >= p.parts) return;
  const Part l = part_at(p, part);
  int left = l.count, row = (int)((unsigned)l.first / (unsigned)p.granules);
  int q = l.first - row * p.granules;
  // The granules ahead: sequence, row and granule of the next to be loaded, and how many are left.
  // `run` of them (already counted) need nothing looked at: they are wanted and all of them the row's.
  int ab = (int)((unsigned)row / (unsigned)p.rows), aj = row - ab * p.rows, aq = q, aleft = left, run = 0;
  const T *ax, *ap;
  bool wanted = true;                      // (of the first row: for the first granules)
  auto at_row = [&]() {
    ax = row_at<T>(a, ab, aj);
    ap = ax - shift_of(ax) + (long long)aq * G::kLogits + lane * G::kVec;
  };
  at_row();
  uint4 ahead[kDepth][2];
  auto slow_load = [&](uint4 (&to)[2]) {
    if (aleft == 0) return;
    if (aq == p.granules) {
      aq = 0;
      if (++aj == p.rows) aj = 0, ++ab;
      at_row();
      wanted = needed(a, ab, aj);
    }
    if (wanted)
#pragma unroll
      for (int v = 0; v < 2; ++v) to[v] = edge_vec<false>(ax, ap - ax + v * 32 * G::kVec, a.V);
    ap += G::kLogits;
    ++aq, --aleft;
    run = wanted && aq > 0 ? max(0, min(aleft, p.granules - 2 - aq)) : 0;
    aq += run, aleft -= run;
  };
  auto load = [&](uint4 (&to)[2]) {
    if (run > 0) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const T* at = ap + v * 32 * G::kVec;
        if (in_bounds(&g_err_lp, at >= ax && at + G::kVec <= ax + a.V)) to[v] = load_inner<false>(at);
      }
      ap += G::kLogits;
      --run;
    } else {
      slow_load(to);
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(ahead[i]);
  wanted = needed(a, ab, aj);
  if (!wanted) aq -= run, aleft += run, run = 0;
  while (left > 0) {
    // ---- this warp's granules of a row
    const int b = (int)((unsigned)row / (unsigned)p.rows), j = row - b * p.rows;
    const float c = scale_of(a.scale ? a.scale[b] : 1.0f) * kLog2e;
    const bool read = needed(a, b, j);     // (then it was loaded)
    Reference ref;
    ref.start();
    int first = 0;                         // the first of this lane's granules that holds m
    unsigned long long z2 = 0;
    const int q0 = q, q1 = q + left < p.granules ? q + left : p.granules;
#pragma unroll kDepth
    for (; q < q1; ++q) {
      float f[G::kPer], top, least;
      widen(ahead[0][0], (const T*)nullptr, f);
      widen(ahead[0][1], (const T*)nullptr, f + G::kVec);
      range(ahead[0][0], ahead[0][1], (const T*)nullptr, f, &top, &least);
#pragma unroll
      for (int i = 0; i + 1 < kDepth; ++i) {
        ahead[i][0] = ahead[i + 1][0];
        ahead[i][1] = ahead[i + 1][1];
      }
      load(ahead[kDepth - 1]);
      if (!read) continue;
      if (top > ref.m) {                   // seldom after the first granules
        const float s = ref.raise(top, c);
        z2 = mul2(z2, pair(s, s));         // (a NaN stays)
        first = q;
      }
      if (ref.m != -INFINITY || top != top) {
        ref.terms(f, c, [&](int, float w0, float w1) { z2 = add2(z2, pair(w0, w1)); });
      }
    }
    left -= q1 - q0;
    // ---- their statistics
    float z0, z1;
    unpair(z2, &z0, &z1);
    const Row st = warp_merge(Row{ref.m, ref.m == -INFINITY ? z0 + z1 : (z0 + z1) * ref.settled(c),
                                  ref.m == -INFINITY ? q0 : first}, c);
    if (lane == 0 && in_bounds(&g_err_lp, b < a.B && part < p.parts))
      p.stats[(long long)row + part] = make_float4(st.m, st.z, __int_as_float(st.q), 0.0f);
    if (q == p.granules) q = 0, ++row;
  }
}

// Without drafts: the rows' statistics, and the race of each, in one pass.
template <typename T>
__global__ void __launch_bounds__(kThreads, draw_ctas(sizeof(T) == 2)) gdn_verify_draw_rows_kernel(
    GdnVerifyArgs a, Plan p) {
  using G = Granule<T>;
  constexpr int kVec = G::kVec;
  const int lane = threadIdx.x & 31, part = blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_wait();                              // (nothing is read before)
  pdl_trigger();
  if (part >= p.parts) return;
  const Part l = part_at(p, part);
  int left = l.count, b = (int)((unsigned)l.first / (unsigned)p.granules);
  int q = l.first - b * p.granules;
  // the granule ahead: sequence and granule of the next to be loaded
  int aleft = left, ab = b, aq = q;
  const T* ax = row_at<T>(a, ab, 0);
  // 0: nothing, 1: the row (greedy), 2: its clocks too (of the first row: for the first granule)
  int wanted = 2;
  uint4 ahead[2];
  float clock[2][kVec];
  auto load = [&](int v) {                 // its v-th vectors
    if (aleft == 0 || wanted == 0) return;
    const long long i = (long long)aq * G::kLogits - shift_of(ax) + (v * 32 + lane) * kVec;
    const bool inner = aq > 0 && aq + 2 < p.granules;      // all of it the row's
    if (inner && in_bounds(&g_err_lp, i >= 0 && i + kVec <= a.V)) ahead[v] = load_inner(ax + i);
    else ahead[v] = edge_vec<true>(ax, i, a.V);
    if (wanted == 1) return;               // (128 greedy rows of 151936 in bf16 22.0 us, so 15.9)
    const float* e = a.clocks + (long long)ab * a.V + i;
    if (inner && (reinterpret_cast<uintptr_t>(e) & 15) == 0) {
#pragma unroll
      for (int k = 0; k < kVec; k += 4) widen(load_inner(e + k), (const float*)nullptr, clock[v] + k);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) clock[v][k] = i + k >= 0 && i + k < a.V ? e[k] : 0.0f;
    }
  };
  auto look = [&]() {
    const float given = a.scale ? a.scale[ab] : 1.0f;
    wanted = given == INFINITY ? 1 : in_range(given) ? 2 : 0;
  };
  auto advance = [&]() {
    if (aleft == 0 || --aleft == 0) return;
    if (++aq == p.granules) {
      aq = 0;
      ax = row_at<T>(a, ++ab, 0);
      look();
    }
  };
  load(0);
  load(1);
  advance();
  look();
  while (left > 0) {
    // ---- this warp's granules of a row
    const float given = a.scale ? a.scale[b] : 1.0f, scale = scale_of(given), c = scale * kLog2e;
    const bool read = takes_part(given), races = given != INFINITY;
    Reference ref;
    ref.start();
    const T* x = row_at<T>(a, b, 0);
    Race<T> race{x, nullptr, a.clocks + (long long)b * a.V, -INFINITY, 0.0f, c, 0.0f, scale, -1,
                 0.0f, -1};
    int first = 0;                         // greedy: the first granule that holds the largest
    unsigned long long z2 = 0;
    const int q0 = q, q1 = q + left < p.granules ? q + left : p.granules;
    for (; q < q1; ++q) {
      float f[G::kPer], e[G::kPer], w[G::kPer], top, least;
      widen(ahead[0], (const T*)nullptr, f);
      widen(ahead[1], (const T*)nullptr, f + kVec);
      range(ahead[0], ahead[1], (const T*)nullptr, f, &top, &least);
#pragma unroll
      for (int k = 0; k < G::kPer; ++k) e[k] = clock[k / kVec][k % kVec];
      load(0);
      load(1);
      advance();
      if (!read) continue;
      // one reference for the warp, so that its lanes' races compare
      if (__any_sync(0xffffffffu, top > ref.m)) {        // seldom after the first granules
        const float s = ref.raise(warp_max(top > ref.m ? top : ref.m), c);
        z2 = mul2(z2, pair(s, s));         // (a NaN stays)
        race.best *= s;
        race.mx = ref.m;
        first = q;
      }
      if (ref.m == -INFINITY && !(top != top)) {
#pragma unroll
        for (int k = 0; k < G::kPer; ++k) w[k] = 0.0f;
      } else {
        ref.terms(f, c, [&](int k, float w0, float w1) {
          w[k] = w0, w[k + 1] = w1;
          z2 = add2(z2, pair(w0, w1));
        });
      }
      if (races) {
        const int i0 = q * G::kLogits - shift_of(x) + lane * kVec;
        race.offer(w, e, [&](int k) { return i0 + k / kVec * 32 * kVec + k % kVec; });
      }
    }
    left -= q1 - q0;
    // ---- what they come to
    float z0, z1;
    unpair(z2, &z0, &z1);
    float z = warp_sum(z0 + z1);
    if (ref.m != -INFINITY) {
      const float s = ref.settled(c);
      z *= s;
      race.best *= s;
    }
    if (lane == 0 && in_bounds(&g_err_lp, b < a.B && part < p.parts))
      p.stats[(long long)b + part] =
          races ? make_float4(race.mx, z, __int_as_float(race.at), race.best)
                : make_float4(race.mx, z, __int_as_float(race.mx == -INFINITY ? q0 : first), 0.0f);
    if (q == p.granules) q = 0, ++b;
  }
}

// The parts of a row on the line: the first, and how many.
__device__ __forceinline__ Part parts_of(const Plan& p, int row) {
  const int c0 = part_of(p, row * p.granules);
  return Part{c0, part_of(p, row * p.granules + p.granules - 1) - c0 + 1};
}

constexpr int kAtOnce = 4;                 // entries of a lane on the way
// Entries k0 + lane, + 32, ... of the parts of a row (none: as of no logits).
__device__ __forceinline__ void entries_of(const Plan& p, int row, const Part& parts, int k0,
                                           float4 (&v)[kAtOnce]) {
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int at = k0 + 32 * k + (threadIdx.x & 31);
    const bool some = at < parts.count &&
                      in_bounds(&g_err_lp, parts.first >= 0 && parts.first + at < p.parts);
    v[k] = some ? p.stats[(long long)row + parts.first + at]
                : make_float4(-INFINITY, 0.0f, __int_as_float(0x7fffffff), 0.0f);
  }
}
// The statistics of a row from its parts' (the whole warp); v keeps the first entries.
__device__ __forceinline__ Row row_of(const Plan& p, int row, const Part& parts, float c,
                                      float4 (&v)[kAtOnce]) {
  Row st{-INFINITY, 0.0f, 0x7fffffff};
  for (int k0 = 32 * kAtOnce; k0 < parts.count; k0 += 32 * kAtOnce) {
    entries_of(p, row, parts, k0, v);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) st = merge(st, Row{v[k].x, v[k].y, __float_as_int(v[k].z)}, c);
  }
  entries_of(p, row, parts, 0, v);
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) st = merge(st, Row{v[k].x, v[k].y, __float_as_int(v[k].z)}, c);
  return warp_merge(st, c);
}

// The first of a granule's logits that equals m (the whole warp).
template <typename T>
__device__ __forceinline__ int first_equal(const T* x, int V, int q, float m) {
  constexpr int kVec = Granule<T>::kVec;
  const long long at = (long long)q * Granule<T>::kLogits - shift_of(x);
  int id = 0x7fffffff;
  uint4 u[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) u[v] = edge_vec<false>(x, at + (v * 32 + (int)(threadIdx.x & 31)) * kVec, V);
#pragma unroll
  for (int v = 1; v >= 0; --v) {
    const long long i = at + (v * 32 + (int)(threadIdx.x & 31)) * kVec;
    float f[kVec];
    widen(u[v], (const T*)nullptr, f);
#pragma unroll
    for (int k = kVec - 1; k >= 0; --k)
      if (i + k >= 0 && i + k < V && f[k] == m) id = (int)(i + k);
  }
  return (int)__reduce_min_sync(0xffffffffu, (unsigned)id);
}

// Without drafts: joins a sequence's parts, a warp a sequence.
template <typename T>
__global__ void __launch_bounds__(32) gdn_verify_draw_kernel(GdnVerifyArgs a, Plan p) {
  const int b = blockIdx.x, lane = threadIdx.x;
  const float given = a.scale ? a.scale[b] : 1.0f;
  if (!takes_part(given)) return pdl_wait();           // (see the race's)
  const bool greedy = given == INFINITY;
  const float scale = scale_of(given), c = scale * kLog2e;
  const T* x = row_at<T>(a, b, 0);
  const Part parts = parts_of(p, b);
  float4 v[kAtOnce];
  pdl_wait();
  pdl_trigger();
  const Row st = row_of(p, b, parts, c, v);
  int token = -1;
  const bool dead = !(st.z > 0.0f);        // 0 or NaN: no distribution
  if (!dead && greedy) {
    token = first_equal(x, a.V, st.q, st.m);
  } else if (!dead) {
    Race<T> race{x, nullptr, a.clocks + (long long)b * a.V, st.m, 0.0f, c, 0.0f, scale, -1, 0.0f, -1};
    for (int k0 = 0; k0 < parts.count; k0 += 32 * kAtOnce) {
      if (k0 > 0) entries_of(p, b, parts, k0, v);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)    // to the row's reference
        race.join(v[k].w > 0.0f ? v[k].w * ptx::ex2_approx((v[k].x - st.m) * c) : 0.0f,
                  __float_as_int(v[k].z));
    }
    token = race.at;
  }
  if (lane > 0 || !in_bounds(&g_err_lp, token < a.V)) return;
  a.tokens[b] = token;
  a.accepted[b] = 0;
  if (a.logprobs)
    a.logprobs[b] = token >= 0 ? (ld_elem(x + token) - st.m) * scale - kLn2 * log2f(st.z) : 0.0f;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kRaceCtasPerSm) gdn_verify_race_kernel(GdnVerifyArgs a,
                                                                                  Plan p) {
  using G = Granule<T>;
  constexpr int kVec = G::kVec;
  __shared__ Row s_row[kMaxRows];
  __shared__ int s_arg[kGdnMaxDrafts + 1];            // greedy: the rows' largest
  __shared__ int s_refused;
  __shared__ int s_id[kGdnMaxDrafts];                 // the drafts, and their logits
  __shared__ float s_x[kGdnMaxDrafts];
  __shared__ float s_best[kWarps];
  __shared__ int s_at[kWarps];
  // the last sequences first: their rows were read last
  const int b = a.B - 1 - blockIdx.x / p.pieces, piece = blockIdx.x % p.pieces;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float given = a.scale ? a.scale[b] : 1.0f;
  // (also where all sequences are left out this grid ends behind the rows', as the kernel after it,
  // which may write what they read and use the workspace again, waits for this one alone)
  if (!takes_part(given)) return pdl_wait();
  const bool greedy = given == INFINITY;
  if (greedy && piece > 0) return;         // (piece 0 waits)
  const float scale = scale_of(given), c = scale * kLog2e;
  const int n = drafts_of(a, b);
  if (threadIdx.x == 0) {
    s_refused = n;
    if (piece == 0 && n < a.T && a.ids[(long long)b * a.T + n] >= a.V)
      atomicOr(&g_err_lp, kErrIndex);
  }
  // ---- what the decisions need of the inputs
  const int t = threadIdx.x;
  int id = -1;
  float u = 0.0f, xi = 0.0f, yi = 0.0f;
  if (t < n) {
    id = a.ids[(long long)b * a.T + t];
    u = a.accept_u[(long long)b * a.T + t];
    xi = ld_elem(row_at<T>(a, b, t) + id);
    if (a.draft) yi = ld_elem(row_at<T>(a, b, a.T + 1 + t) + id);
    s_id[t] = id, s_x[t] = xi;
  }
  // (a warp's first row, whose parts are known)
  const int rows = n + 1 + (a.draft ? n : 0);
  auto row_of_sequence = [&](int i) { return i <= n ? i : a.T + 1 + i - n - 1; };
  Part parts = parts_of(p, b * p.rows + row_of_sequence(min(warp, rows - 1)));
  pdl_wait();
  pdl_trigger();
  // ---- the rows' statistics, a warp a row
  for (int i = warp; i < rows; i += kWarps) {
    const int j = row_of_sequence(i), row = b * p.rows + j;
    float4 v[kAtOnce];
    if (i >= kWarps) parts = parts_of(p, row);
    const Row st = row_of(p, row, parts, c, v);
    if (lane == 0) s_row[j] = st;
    if (greedy && j <= a.T) {
      const int arg = first_equal(row_at<T>(a, b, j), a.V, st.q, st.m);
      if (lane == 0) s_arg[j] = arg;
    }
  }
  __syncthreads();
  auto dead = [&](int j) { return !(s_row[j].z > 0.0f); };    // 0 or NaN: no distribution
  // ---- the drafts
  if (t < n) {
    bool good = !dead(t);
    if (good && greedy) {
      good = id == s_arg[t];
    } else if (good) {
      const Row& px = s_row[t];
      float e = (xi - px.m) * c, size = fabsf(e), z = px.z;
      if (a.draft) {
        const Row& py = s_row[a.T + 1 + t];
        // q = 0: accepted unless p = 0 too
        const float ey = (yi - py.m) * c;
        e -= ey;
        size = fmaxf(size, fabsf(ey));
        z /= py.z;
        good = !dead(a.T + 1 + t);
      }
      if (good && xi == -INFINITY) {
        good = false;
      } else if (good) {
        const float r = ptx::ex2_approx(e) / z;
        good = u < r;
        // near the border, or where the exponents are rounded by much: in 64 bits
        if (fabsf(u - r) <= r * 0x1p-14f || !(size < 64.0f)) {
          double far = (double)xi - (double)px.m;
          if (a.draft)
            far = yi == -INFINITY ? (double)INFINITY : difference_of(xi, px.m, yi, s_row[a.T + 1 + t].m);
          good = (double)u < exp(far * (double)scale) / (double)z;
        }
      }
    }
    if (!good) atomicMin(&s_refused, t);
  }
  __syncthreads();
  const int accepted = s_refused, last_draft = accepted < n ? s_id[accepted] : -1;
  const bool refused = accepted < n;
  const int yj = a.T + 1 + accepted;
  const bool hopeless = dead(accepted) || (refused && a.draft && !greedy && dead(yj));
  if (hopeless && piece > 0) return;
  int token = -1;
  float logit = 0.0f;                      // the token's
  if (greedy) {
    token = hopeless ? -1 : s_arg[accepted];
    logit = s_row[accepted].m;
  } else if (!hopeless) {
    // ---- the race over this CTA's slice
    const T* x = row_at<T>(a, b, accepted);
    const T* y = refused && a.draft ? row_at<T>(a, b, yj) : nullptr;
    const float* clocks = a.clocks + (long long)b * a.V;
    Race<T> race{x, y, clocks, s_row[accepted].m, y ? s_row[yj].m : 0.0f, c,
                 y ? s_row[accepted].z / s_row[yj].z : 0.0f, scale,
                 refused && !a.draft ? last_draft : -1, 0.0f, -1};
    const int lo = piece * p.slice, hi = min(a.V, lo + p.slice);
    auto weight = [&](float v, float w) {
      float r = ptx::ex2_approx((v - race.mx) * c);
      if (y) r = fmaf(-race.ratio, ptx::ex2_approx((w - race.my) * c), r);
      return r;
    };
    // x in its own vectors, from lo2 to hi2 (not the row's first logit nor its last two: what is
    // loaded beside a vector of y's is the row's too)
    const int shift = shift_of(x), from = max(lo, 1), to = min(hi, a.V - 2);
    const int lo2 = min(hi, from + (-(from + shift) & (kVec - 1)));
    const int hi2 = max(lo2, to - ((to + shift) & (kVec - 1)));
    const bool wide_y = !y || shift_of(y) == shift;
    const bool wide_e = (reinterpret_cast<uintptr_t>(clocks + lo2) & 15) == 0;
    auto vectors = [&](auto all_wide) {    // all_wide: y's and the clocks' vectors lie as x's do
      constexpr bool kWide = decltype(all_wide)::value;
      const bool odd = !kWide && !wide_y && (reinterpret_cast<uintptr_t>(y + lo2) & 2);
      constexpr int kWords = kWide ? 4 : 5, kAhead = kWide ? 2 : 1;
      uint4 ux[kAhead];
      uint32_t uy[kAhead][kWords];
      float ue[kAhead][kVec];
      auto fetch = [&](int k, int i) {
        if (i >= hi2 || !in_bounds(&g_err_lp, i >= 1 && i + kVec + 2 <= a.V)) return;
        ux[k] = load_inner<false>(x + i);
        if (y && (kWide || wide_y)) {
          const uint4 u = load_inner<false>(y + i);
          uy[k][0] = u.x, uy[k][1] = u.y, uy[k][2] = u.z, uy[k][3] = u.w;
        } else if (y) {
          const uint32_t* at =
              reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(y + i) & ~(uintptr_t)3);
#pragma unroll
          for (int q = 0; q < kWords; ++q) uy[k][q] = at[q];
        }
        if (kWide || wide_e) {
#pragma unroll
          for (int q = 0; q < kVec; q += 4)
            widen(load_inner(clocks + i + q), (const float*)nullptr, ue[k] + q);
        } else {
#pragma unroll
          for (int q = 0; q < kVec; ++q) ue[k][q] = clocks[i + q];
        }
      };
      constexpr int kStride = kThreads * kVec;
      int i = lo2 + (int)threadIdx.x * kVec;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) fetch(k, i + k * kStride);
      for (; i - lane * kVec < hi2; i += kAhead * kStride) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int at = i + k * kStride;
          float v[kVec], w[kVec], e[kVec];
          widen(ux[k], x, v);
          if (odd) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              uy[k][q] = __funnelshift_r(uy[k][q], uy[k][kWords - 4 + q], 16);
          }
          widen(make_uint4(uy[k][0], uy[k][1], uy[k][2], uy[k][3]), x, w);
#pragma unroll
          for (int q = 0; q < kVec; ++q) e[q] = ue[k][q];
          fetch(k, at + kAhead * kStride);
#pragma unroll
          for (int q = 0; q < kVec; ++q) {
            w[q] = weight(v[q], w[q]);
            if (at >= hi2) w[q] = e[q] = 0.0f;
          }
          race.offer(w, e, [&](int q) { return at + q; });
        }
      }
      if (warp == 0) {                     // the slice's logits before and behind them, up to nine each
        const int at = lane < 16 ? lo + lane : hi2 + lane - 16;
        float w[1] = {0.0f}, e[1] = {0.0f};
        if (at < (lane < 16 ? lo2 : hi) && in_bounds(&g_err_lp, at >= 0 && at < a.V))
          w[0] = weight(ld_elem(x + at), y ? ld_elem(y + at) : 0.0f), e[0] = clocks[at];
        race.offer(w, e, [&](int) { return at; });
      }
    };
    // 16-bit logits are read so whatever the others' alignment: y's vectors as the words that hold
    // them, clocks one by one (64 sequences of 4 drafts over 151669 logits element by element 62 us,
    // so 57).  32-bit ones element by element: 16 of 7 drafts over 151669 26.5 us, so 27
    // to 28.
    if (wide_y && wide_e) {
      vectors(std::true_type{});
    } else if constexpr (sizeof(T) == 2) {
      vectors(std::false_type{});
    } else {
      constexpr int kN = 4, kAhead = 2;    // a lane's elements, 32 apart, and how often
      float v[kAhead][kN], w[kAhead][kN], e[kAhead][kN];
      auto fetch = [&](int d, int i0) {
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const int i = i0 + 32 * k + lane;
          const bool in = i < hi && in_bounds(&g_err_lp, i >= 0 && i < a.V);
          v[d][k] = in ? ld_elem(x + i) : -INFINITY;
          w[d][k] = in && y ? ld_elem(y + i) : -INFINITY;
          e[d][k] = in ? clocks[i] : 0.0f;
        }
      };
      constexpr int kStride = kThreads * kN;
      int i0 = lo + warp * 32 * kN;
#pragma unroll
      for (int d = 0; d < kAhead; ++d) fetch(d, i0 + d * kStride);
      for (; i0 < hi; i0 += kAhead * kStride) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const int at = i0 + d * kStride;
          float w1[kN], e1[kN];
#pragma unroll
          for (int k = 0; k < kN; ++k) w1[k] = weight(v[d][k], w[d][k]), e1[k] = e[d][k];
          fetch(d, at + kAhead * kStride);
          race.offer(w1, e1, [&](int k) { return at + lane + 32 * k; });
        }
      }
    }
    // ---- the slice's best
    if (lane == 0) s_best[warp] = race.best, s_at[warp] = race.at;
    __syncthreads();
    if (warp > 0) return;
    race.best = 0.0f, race.at = -1;
    race.join(lane < kWarps ? s_best[lane] : 0.0f, lane < kWarps ? s_at[lane] : -1);
    if (race.at >= 0 && in_bounds(&g_err_lp, race.at < a.V)) logit = ld_elem(x + race.at);   // (in L1)
    // ---- the last CTA of the sequence joins the slices
    if (p.pieces > 1) {
      float4* slices = p.best + (long long)b * p.pieces;
      int last = 0;
      if (lane == 0) {
        __stcg(&slices[piece], make_float4(race.best, __int_as_float(race.at), logit, 0.0f));
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;\n"
                     : "=r"(last) : "l"(&p.done[b]) : "memory");
      }
      if (__shfl_sync(0xffffffffu, last, 0) != p.pieces - 1) return;
      __threadfence();                     // (lane 0 acquired for the others)
      __syncwarp();
      race.best = 0.0f, race.at = -1;
      for (int k0 = 0; k0 < p.pieces; k0 += 32 * kAtOnce) {
        float4 r[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int slice = k0 + 32 * k + lane;
          r[k] = slice < p.pieces ? __ldcg(&slices[slice])
                                  : make_float4(0.0f, __int_as_float(-1), 0.0f, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          race.join(r[k].x, __float_as_int(r[k].y));
          const uint32_t who =
              __ballot_sync(0xffffffffu, race.at >= 0 && __float_as_int(r[k].y) == race.at);
          if (who) logit = __shfl_sync(0xffffffffu, r[k].z, __ffs(who) - 1);
        }
      }
    }
    token = race.at;
    if (token < 0 && refused) token = last_draft, logit = s_x[accepted];   // p = q but for rounding
  }
  if (warp > 0) return;
  // ---- what the sequence gets
  for (int k = lane; k <= a.T; k += 32) {
    const int given_id = k < accepted ? s_id[k] : k == accepted ? token : -1;
    const long long to = (long long)b * (a.T + 1) + k;
    if (!in_bounds(&g_err_lp, given_id < a.V)) continue;
    a.tokens[to] = given_id;
    if (a.logprobs) {
      float lp = 0.0f;
      if (given_id >= 0)
        lp = scaled_difference(k < accepted ? s_x[k] : logit, s_row[k].m, scale) -
             kLn2 * log2f(s_row[k].z);   // (an accepted draft's logit may be far below)
      a.logprobs[to] = lp;
    }
  }
  if (lane == 0) a.accepted[b] = accepted;
}

constexpr int kRaceCtas = 152 * kRaceCtasPerSm, kLeastSlice = 2048, kLeastGranules = 2;
// Rows that are one slice: a second one costs a join (one request of 3 drafts over 4096 logits 9.9 us in
// two slices, 8.6 in one; over 8192 9.8 in four, 9.6 in one).
constexpr int kOneSlice = 4096;

Plan plan_of(int B, int T, int V, int bf16, bool draft) {
  Plan p = {};
  p.granules = granules_of(V, bf16);
  p.rows = T + 1 + (draft ? T : 0);
  const int total = p.granules * p.rows * B;
  // a few granules a part: the second pass joins what the parts of a row leave
  const int most = (total + kLeastGranules - 1) / kLeastGranules;
  const int warps = 152 * kWarps * (T ? kCtasPerSm : draw_ctas(bf16));
  p.parts = most < warps ? most : warps;
  p.each = total / p.parts;
  p.more = total % p.parts;
  // slices: one round of CTAs
  int pieces = kRaceCtas / B;
  const int pieces_most = V <= kOneSlice ? 1 : (V + kLeastSlice - 1) / kLeastSlice;
  pieces = pieces < 1 ? 1 : pieces < pieces_most ? pieces : pieces_most;
  p.slice = ((V + pieces - 1) / pieces + 15) & ~15;
  p.pieces = (V + p.slice - 1) / p.slice;
  // room for the slices of any smaller batch and vocabulary too (456 / B goes down in steps), so that
  // what a larger call needs is never less
  p.room = T ? std::min((long long)std::max(kRaceCtas, B), (long long)B * pieces_most) : 0;
  return p;
}
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
size_t stats_bytes(const Plan& p, int B) {
  return up(sizeof(float4) * ((size_t)p.rows * B + p.parts));
}
size_t best_bytes(const Plan& p) { return up(sizeof(float4) * (size_t)p.room); }

template <typename T>
cudaError_t launch(const GdnVerifyArgs& a, const Plan& p, cudaStream_t stream) {
  const int grid = (p.parts + kWarps - 1) / kWarps;
  // (set up while the kernel before ends: one request 14.2 -> 11.2 us in a stream)
  const cudaError_t e =
      launch_pdl(true, a.T ? gdn_verify_rows_kernel<T> : gdn_verify_draw_rows_kernel<T>,
                 dim3((unsigned)grid), dim3(kThreads), 0, stream, a, p);
  if (e != cudaSuccess) return e;
  if (a.T == 0)
    return launch_pdl(true, gdn_verify_draw_kernel<T>, dim3((unsigned)a.B), dim3(32), 0, stream, a, p);
  return launch_pdl(true, gdn_verify_race_kernel<T>, dim3((unsigned)(p.pieces * a.B)),
                    dim3(kThreads), 0, stream, a, p);
}

}  // namespace verify
}  // namespace

size_t gdn_verify_tokens_bytes(int B, int T, int V, int bf16, int draft) {
  const verify::Plan p = verify::plan_of(B, T, V, bf16, draft);
  return verify::stats_bytes(p, B) + verify::best_bytes(p) + (T ? verify::up(sizeof(int) * (size_t)B) : 0);
}

cudaError_t gdn_launch_verify_tokens(const GdnVerifyArgs& a, cudaStream_t stream) {
  verify::Plan p = verify::plan_of(a.B, a.T, a.V, a.bf16, a.draft != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.stats = reinterpret_cast<float4*>(ws);
  p.best = reinterpret_cast<float4*>(ws + verify::stats_bytes(p, a.B));
  p.done = reinterpret_cast<int*>(ws + verify::stats_bytes(p, a.B) + verify::best_bytes(p));
  return a.bf16 ? verify::launch<__nv_bfloat16>(a, p, stream) : verify::launch<float>(a, p, stream);
}
