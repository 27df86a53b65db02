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
// pair that matters, which L2 still holds where the batch is small: a CTA a slice, the last CTA of a
// sequence joins the slices.  An element takes part only if w > best E, so there is a division
// where the best changes and none elsewhere, and p's normaliser cancels: w = e^.. - e^.. (z_p / z_q).
// The decisions are compared in 32 bits and, where two are within 2^-16 of each other, again in 64.
// Part of logprobs.cu, whose error word it uses.
#pragma once

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
constexpr int kCtasPerSm = 4, kParts = 152 * kCtasPerSm * kWarps;
constexpr int kMaxRows = 2 * kGdnMaxDrafts + 1;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMost = 18446744073709551616.0f;       // 2^64: scales lie within it and its inverse
constexpr float kClose = 1.0f - 0x1p-16f;

struct Plan {
  long long total;                         // granules of all rows
  int granules;                            // of a row
  int rows;                                // of a sequence: T + 1 of the target, then the draft's
  int parts;                               // equal parts of the line, a warp's each
  int pieces;                              // slices of a sequence's race
  int slice;                               // logits of a slice
  float4* stats;                           // [row + part]: m, z, granule of the largest
  float2* best;                            // [B][pieces]: w / E and its index
  int* done;                               // [B]
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
__device__ __forceinline__ Row warp_merge(Row a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = merge(a, Row{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.z, o),
                     __shfl_xor_sync(0xffffffffu, a.q, o)}, c);
  return a;
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

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) gdn_verify_rows_kernel(GdnVerifyArgs a,
                                                                              Plan p) {
  using G = Granule<T>;
  constexpr int kDepth = 2;                // granules on the way
  const int lane = threadIdx.x & 31, part = blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_trigger();
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.B; b += gridDim.x * kThreads) p.done[b] = 0;
  if (part >= p.parts) return;
  const long long start = p.total * part / p.parts;
  int left = (int)(p.total * (part + 1) / p.parts - start);
  const long long row0 = start / p.granules;
  long long row = row0;                    // of all sequences
  int q = (int)(start - row * p.granules); // granule of the row
  int b = (int)(row / p.rows), j = (int)(row - (long long)b * p.rows);
  // the granules ahead: the sequence, row and granule of the next to be loaded
  int ab = b, aj = j, aq = q, aleft = left;
  const T* ax = row_at<T>(a, ab, aj);
  const T* ap = ax - shift_of(ax) + (long long)aq * G::kLogits + lane * G::kVec;
  bool wanted = true;                      // (the first row is read before that is known)
  uint4 ahead[kDepth][2];
  auto load = [&](uint4 (&to)[2]) {
    if (aleft <= 0) return;
    if (wanted) {
      if (aq > 0 && aq + 2 < p.granules) { // all of it the row's
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const T* at = ap + v * 32 * G::kVec;
          if (in_bounds(&g_err_lp, at >= ax && at + G::kVec <= ax + a.V))
            to[v] = load_inner<false>(at);
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) to[v] = load_vec<false>(ax, ap - ax + v * 32 * G::kVec, a.V);
      }
    }
    --aleft;
    ap += G::kLogits;
    if (++aq == p.granules) {
      aq = 0;
      if (++aj == p.rows) aj = 0, ++ab;
      if (aleft > 0) {
        const int n = drafts_of(a, ab);
        wanted = takes_part(a.scale ? a.scale[ab] : 1.0f) && (aj <= a.T ? aj <= n : aj - a.T - 1 < n);
        ax = row_at<T>(a, ab, aj);
        ap = ax - shift_of(ax) + lane * G::kVec;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(ahead[i]);
  while (left > 0) {
    // ---- this warp's granules of a row
    const float scale = a.scale ? a.scale[b] : 1.0f;
    const float c = scale_of(scale) * kLog2e;
    const unsigned long long c2 = pair(c, c);
    float m = -INFINITY;
    int first = 0;                         // the first of this lane's granules that holds m
    unsigned long long z2 = 0;
    const int q0 = q, q1 = q + left < p.granules ? q + left : p.granules;
    bool read = takes_part(scale);
    if (row != row0) {       // (as decided when the row was loaded)
      const int n = drafts_of(a, b);
      read = read && (j <= a.T ? j <= n : j - a.T - 1 < n);
    }
#pragma unroll kDepth
    for (; q < q1; ++q) {
      if (read) {
        float f[G::kPer], top, least;
        widen(ahead[0][0], (const T*)nullptr, f);
        widen(ahead[0][1], (const T*)nullptr, f + G::kVec);
        range(ahead[0][0], ahead[0][1], (const T*)nullptr, f, &top, &least);
        if (top > m) {                     // seldom after the first granules
          const float s = ptx::ex2_approx((m - top) * c);
          z2 = mul2(z2, pair(s, s));       // (0 from m = -inf; a NaN stays)
          m = top;
          first = q;
        }
        if (m != -INFINITY || top != top) {
          const unsigned long long minus_m = pair(-m, -m);
#pragma unroll
          for (int e = 0; e < G::kPer; e += 2) {
            float t0, t1;
            unpair(mul2(add2(pair(f[e], f[e + 1]), minus_m), c2), &t0, &t1);
            z2 = add2(z2, pair(ptx::ex2_approx(t0), ptx::ex2_approx(t1)));
          }
        }
      }
#pragma unroll
      for (int i = 0; i + 1 < kDepth; ++i) {
        ahead[i][0] = ahead[i + 1][0];
        ahead[i][1] = ahead[i + 1][1];
      }
      load(ahead[kDepth - 1]);
    }
    left -= q1 - q0;
    // ---- their statistics
    float z0, z1;
    unpair(z2, &z0, &z1);
    const Row st = warp_merge(Row{m, z0 + z1, m == -INFINITY ? q0 : first}, c);
    if (lane == 0 && in_bounds(&g_err_lp, b < a.B && part < kParts))
      p.stats[row + part] = make_float4(st.m, st.z, __int_as_float(st.q), 0.0f);
    if (q == p.granules) {
      q = 0;
      ++row;
      if (++j == p.rows) j = 0, ++b;
    }
  }
}

// Is (v, i) before (w, j) in the race?  The larger, then the lower index.
__device__ __forceinline__ bool beats(float v, int i, float w, int j) {
  return v > w || (v == w && i < j);
}

// The race's elements of one sequence, as each thread of the second kernel needs them.
template <typename T>
struct Race {
  const T* x;                              // the target's row
  const T* y;                              // the draft's, or NULL
  const float* clocks;
  float mx, my, c, ratio;                  // ratio: z_p / z_q
  double scale;
  int never;                               // the refused draft where q is all on it, or -1
  float best;
  int at;

  __device__ __forceinline__ void offer(float w, float e, int i) {
    if (!(w > best * e)) return;           // seldom after the first elements
    const float r = __fdiv_rn(w, e);
    if (e > 0.0f && i != never && r > best) best = r, at = i;
  }
  // w / E in 64 bits
  __device__ __forceinline__ double exactly(int i) const {
    double w = exp(((double)ld_elem(x + i) - (double)mx) * scale);
    if (y) w -= exp(((double)ld_elem(y + i) - (double)my) * scale) * (double)ratio;
    return w / (double)clocks[i];
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) gdn_verify_race_kernel(GdnVerifyArgs a, Plan p) {
  using G = Granule<T>;
  __shared__ Row s_row[kMaxRows];
  __shared__ int s_arg[kGdnMaxDrafts + 1];            // greedy: the rows' largest
  __shared__ int s_refused, s_last;
  __shared__ float s_best[kWarps];
  __shared__ int s_at[kWarps];
  __shared__ int s_winner;
  const int b = blockIdx.x / p.pieces, piece = blockIdx.x - b * p.pieces;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float given = a.scale ? a.scale[b] : 1.0f;
  if (!takes_part(given)) return;
  const bool greedy = given == INFINITY;
  if (greedy && piece > 0) return;
  const float scale = scale_of(given), c = scale * kLog2e;
  const int n = drafts_of(a, b);
  if (threadIdx.x == 0) {
    s_refused = n;
    if (piece == 0 && n < a.T && a.ids[(long long)b * a.T + n] >= a.V)
      atomicOr(&g_err_lp, kErrIndex);
  }
  pdl_wait();
  // ---- the rows' statistics, a warp a row
  for (int i = warp; i < n + 1 + (a.draft ? n : 0); i += kWarps) {
    const int j = i <= n ? i : a.T + 1 + i - n - 1;    // row of the sequence
    const long long row = (long long)b * p.rows + j;
    const long long x0 = row * p.granules, x1 = x0 + p.granules - 1;
    const int c0 = (int)(((x0 + 1) * p.parts - 1) / p.total);
    const int pieces = (int)(((x1 + 1) * p.parts - 1) / p.total) - c0 + 1;
    Row st{-INFINITY, 0.0f, 0x7fffffff};
    for (int k = lane; k < pieces; k += 32) {
      if (!in_bounds(&g_err_lp, c0 >= 0 && c0 + k < kParts)) break;
      const float4 v = p.stats[row + c0 + k];
      st = merge(st, Row{v.x, v.y, __float_as_int(v.z)}, c);
    }
    st = warp_merge(st, c);
    if (lane == 0) s_row[j] = st;
    if (greedy && j <= a.T) {              // the first of the granule's logits that is the largest
      const T* x = row_at<T>(a, b, j);
      const long long at = (long long)st.q * G::kLogits - shift_of(x);
      int id = 0x7fffffff;
      for (int e = lane; e < G::kLogits; e += 32)
        if (at + e >= 0 && at + e < a.V && ld_elem(x + at + e) == st.m) id = min(id, (int)(at + e));
      id = (int)__reduce_min_sync(0xffffffffu, (unsigned)id);
      if (lane == 0) s_arg[j] = id;
    }
  }
  __syncthreads();
  auto dead = [&](int j) { return !(s_row[j].z > 0.0f); };    // 0 or NaN: no distribution
  // ---- the drafts
  if ((int)threadIdx.x < n) {
    const int t = threadIdx.x, id = a.ids[(long long)b * a.T + t];
    bool good = !dead(t);
    if (good && greedy) {
      good = id == s_arg[t];
    } else if (good) {
      const T* x = row_at<T>(a, b, t);
      const float u = a.accept_u[(long long)b * a.T + t];
      const Row& px = s_row[t];
      const float xi = ld_elem(x + id);
      float e = (xi - px.m) * c, size = fabsf(e), z = px.z;
      double far = ((double)xi - (double)px.m) * (double)scale;
      if (a.draft) {
        const Row& py = s_row[a.T + 1 + t];
        if (dead(a.T + 1 + t)) {
          good = false;
        } else {
          const float yi = ld_elem(row_at<T>(a, b, a.T + 1 + t) + id);
          // q = 0: accepted unless p = 0 too
          const float ey = (yi - py.m) * c;
          e -= ey;
          size = fmaxf(size, fabsf(ey));
          far -= ((double)yi - (double)py.m) * (double)scale;
          z /= py.z;
        }
      }
      if (good && xi == -INFINITY) {
        good = false;
      } else if (good) {
        const float r = ptx::ex2_approx(e) / z;
        good = u < r;
        // near the border, or where the exponents are rounded by much: in 64 bits
        if (fabsf(u - r) <= r * 0x1p-14f || !(size < 64.0f)) good = (double)u < exp(far) / (double)z;
      }
    }
    if (!good) atomicMin(&s_refused, t);
  }
  __syncthreads();
  const int accepted = s_refused, last_draft = accepted < n ? a.ids[(long long)b * a.T + accepted] : -1;
  const bool refused = accepted < n;
  const int yj = a.T + 1 + accepted;
  const bool hopeless = dead(accepted) || (refused && a.draft && !greedy && dead(yj));
  if (hopeless && piece > 0) return;
  int token = -1;
  if (greedy) {
    token = hopeless ? -1 : s_arg[accepted];
  } else if (!hopeless) {
    // ---- the race over this CTA's slice
    Race<T> race;
    race.x = row_at<T>(a, b, accepted);
    race.y = refused && a.draft ? row_at<T>(a, b, yj) : nullptr;
    race.clocks = a.clocks + (long long)b * a.V;
    race.mx = s_row[accepted].m;
    race.my = race.y ? s_row[yj].m : 0.0f;
    race.ratio = race.y ? s_row[accepted].z / s_row[yj].z : 0.0f;
    race.c = c;
    race.scale = scale;
    race.never = refused && !a.draft ? last_draft : -1;
    race.best = 0.0f;
    race.at = -1;
    const int lo = piece * p.slice, hi = min(a.V, lo + p.slice);
    auto weight = [&](float x, float y) {
      float w = ptx::ex2_approx((x - race.mx) * c);
      if (race.y) w -= ptx::ex2_approx((y - race.my) * c) * race.ratio;
      return w;
    };
    constexpr int kVec = G::kVec;
    const bool aligned =
        ((reinterpret_cast<uintptr_t>(race.x) | reinterpret_cast<uintptr_t>(race.clocks) |
          (race.y ? reinterpret_cast<uintptr_t>(race.y) : 0)) & 15) == 0;
    if (aligned) {                         // (a slice is a multiple of 16 logits)
      int i = lo + (int)threadIdx.x * kVec;
      for (; i + kVec <= hi; i += kThreads * kVec) {
        if (!in_bounds(&g_err_lp, i >= 0 && i + kVec <= a.V)) break;
        const uint4 ux = *reinterpret_cast<const uint4*>(race.x + i);
        const uint4 uy = race.y ? *reinterpret_cast<const uint4*>(race.y + i) : make_uint4(0, 0, 0, 0);
        float x[kVec], y[kVec], e[kVec];
#pragma unroll
        for (int k = 0; k < kVec; k += 4) {
          const uint4 ue = load_inner(race.clocks + i + k);
          widen(ue, (const float*)nullptr, e + k);
        }
        widen(ux, race.x, x);
        widen(uy, race.x, y);
#pragma unroll
        for (int k = 0; k < kVec; ++k) race.offer(weight(x[k], y[k]), e[k], i + k);
      }
      for (; i < hi; ++i)                  // at most one thread's, the row's last logits
        race.offer(weight(ld_elem(race.x + i), race.y ? ld_elem(race.y + i) : 0.0f), race.clocks[i], i);
    } else {
#pragma unroll 4
      for (int i = lo + (int)threadIdx.x; i < hi; i += kThreads) {
        if (!in_bounds(&g_err_lp, i >= 0 && i < a.V)) break;
        race.offer(weight(ld_elem(race.x + i), race.y ? ld_elem(race.y + i) : 0.0f), race.clocks[i], i);
      }
    }
    // ---- the slice's best; of those close to it the best in 64 bits
    auto block_best = [&](float v, int i) {
      for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        const int k = __shfl_xor_sync(0xffffffffu, i, o);
        if (beats(w, k, v, i)) v = w, i = k;
      }
      if (lane == 0) s_best[warp] = v, s_at[warp] = i;
      __syncthreads();
      v = s_best[0], i = s_at[0];
#pragma unroll
      for (int k = 1; k < kWarps; ++k)
        if (beats(s_best[k], s_at[k], v, i)) v = s_best[k], i = s_at[k];
      return make_float2(v, __int_as_float(i));
    };
    __shared__ double s_value[kThreads];
    __shared__ int s_index[kThreads];
    // the best (v, i) of the block's threads; several near it are compared in 64 bits
    auto settle = [&](float v, int i) {
      const float2 top = block_best(v, i);
      const bool near = v > 0.0f && v >= top.x * kClose;
      if (__syncthreads_count(near) < 2) return top;
      s_value[threadIdx.x] = near ? race.exactly(i) : -1.0;             // (rare)
      s_index[threadIdx.x] = i;
      __syncthreads();
      if (threadIdx.x == 0) {
        int w = 0;
        for (int k = 1; k < kThreads; ++k)
          if (s_value[k] > s_value[w] || (s_value[k] == s_value[w] && s_index[k] < s_index[w])) w = k;
        s_winner = w;
      }
      __syncthreads();
      const float2 r = make_float2(top.x, __int_as_float(s_index[s_winner]));
      __syncthreads();
      return r;
    };
    const float2 mine = settle(race.best, race.at);
    // ---- the last CTA of the sequence joins the slices
    if (p.pieces > 1) {
      if (threadIdx.x == 0) {
        p.best[(long long)b * p.pieces + piece] = mine;
        __threadfence();
        s_last = atomicAdd(&p.done[b], 1) == p.pieces - 1;
      }
      __syncthreads();
      if (!s_last) return;
      __threadfence();
      float v = 0.0f;
      int i = -1;
      for (int k = threadIdx.x; k < p.pieces; k += kThreads) {
        const float2 r = __ldcg(&p.best[(long long)b * p.pieces + k]);
        if (beats(r.x, __float_as_int(r.y), v, i)) v = r.x, i = __float_as_int(r.y);
      }
      token = __float_as_int(settle(v, i).y);
    } else {
      token = __float_as_int(mine.y);
    }
    if (token < 0 && refused) token = last_draft;      // p = q but for rounding
  }
  // ---- what the sequence gets
  for (int t = threadIdx.x; t <= a.T; t += kThreads) {
    const int id = t < accepted ? a.ids[(long long)b * a.T + t] : t == accepted ? token : -1;
    const long long to = (long long)b * (a.T + 1) + t;
    if (!in_bounds(&g_err_lp, id < a.V)) continue;
    a.tokens[to] = id;
    if (a.logprobs) {
      float lp = 0.0f;
      if (id >= 0)
        lp = (ld_elem(row_at<T>(a, b, t) + id) - s_row[t].m) * scale - kLn2 * log2f(s_row[t].z);
      a.logprobs[to] = lp;
    }
  }
  if (threadIdx.x == 0) a.accepted[b] = accepted;
}

constexpr int kRaceCtas = 152 * 4, kLeastSlice = 2048;

Plan plan_of(int B, int T, int V, int bf16, bool draft) {
  Plan p = {};
  p.granules = granules_of(V, bf16);
  p.rows = T + 1 + (draft ? T : 0);
  p.total = (long long)p.granules * p.rows * B;
  p.parts = (int)(p.total < kParts ? p.total : kParts);
  int pieces = (kRaceCtas + B - 1) / B;
  const int most = (V + kLeastSlice - 1) / kLeastSlice;
  pieces = pieces < most ? pieces : most;
  p.slice = ((V + pieces - 1) / pieces + 15) & ~15;
  p.pieces = (V + p.slice - 1) / p.slice;
  return p;
}
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
size_t stats_bytes(const Plan& p, int B) {
  return up(sizeof(float4) * ((size_t)p.rows * B + p.parts));
}
size_t best_bytes(const Plan& p, int B) { return up(sizeof(float2) * (size_t)p.pieces * B); }

template <typename T>
cudaError_t launch(const GdnVerifyArgs& a, const Plan& p, cudaStream_t stream) {
  gdn_verify_rows_kernel<T><<<(p.parts + kWarps - 1) / kWarps, kThreads, 0, stream>>>(a, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(true, gdn_verify_race_kernel<T>, dim3((unsigned)(p.pieces * a.B)),
                    dim3(kThreads), 0, stream, a, p);
}

}  // namespace verify
}  // namespace

size_t gdn_verify_tokens_bytes(int B, int T, int V, int bf16, int draft) {
  const verify::Plan p = verify::plan_of(B, T, V, bf16, draft);
  return verify::stats_bytes(p, B) + verify::best_bytes(p, B) + verify::up(sizeof(int) * (size_t)B);
}

cudaError_t gdn_launch_verify_tokens(const GdnVerifyArgs& a, cudaStream_t stream) {
  verify::Plan p = verify::plan_of(a.B, a.T, a.V, a.bf16, a.draft != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.stats = reinterpret_cast<float4*>(ws);
  p.best = reinterpret_cast<float2*>(ws + verify::stats_bytes(p, a.B));
  p.done = reinterpret_cast<int*>(ws + verify::stats_bytes(p, a.B) + verify::best_bytes(p, a.B));
  return a.bf16 ? verify::launch<__nv_bfloat16>(a, p, stream) : verify::launch<float>(a, p, stream);
}
