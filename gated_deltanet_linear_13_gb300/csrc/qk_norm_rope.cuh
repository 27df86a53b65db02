// The norm of query and key heads with their rotation by position, and the write of keys and
// values to the paged cache, in one pass.
//
// Per head vector x of D elements: y = x rsqrt(mean x^2 + eps) w, then each pair (a, b) of its
// first r elements is turned by the angle w_p = position * frequency_p.  The angle is kept as a
// phase in 2^64ths of a turn: position * step_p modulo 2^64 is one 64-bit product, exact for every
// position (in 32 bits an angle of 10^6 radians is off by 0.03); its upper 32 bits, rounded to a float,
// give cos and sin to 2^-26 of a turn.  All in fp32, rounded once to what is stored; an 8-bit cache
// is quantised from the fp32 keys.
//
// L lanes a vector, two runs of eight elements each (16 bytes of bf16): in the half layout a lane's
// runs are the two halves of its pairs, otherwise they are neighbours, so a pair lies in one lane
// either way and a lane with elements to turn has the pairs 8 l .. 8 l + 7.  Halves that are no
// multiple of eight elements meet in shared memory.  A token's cos and sin are made once for all
// its heads, while the first heads are on their way; a lane group takes kHeads heads of a token at
// a time, so that addresses and weights cost once for all of them: what bounds the pass beside
// memory is instructions (each vector finding its own took 228 a vector and 119 us below; this takes 117).
// Measured: 16384 tokens of 24 + 4 + 4 heads of 256 in bf16 into a bf16 cache 89 us (6.0 TB/s read and
// written, 89% of the copy rate), 2501 tokens of 16 + 2 heads of 128 in fp32 11.8 us (latency: four
// rounds of vectors a lane group behind the launch and the angles), 64 tokens 2.8 us, one 2.5: the
// launch.
// Part of kv_cache.cu, whose error word it uses.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kv_cache.cuh"
#include "sm100_ptx.cuh"

using namespace gdn;
using ptx::fma2;
using ptx::mul2;
using ptx::pair;
using ptx::unpair;

namespace {
namespace rope {
constexpr int kThreads = 128;
constexpr int kMaxPairs = 128, kRun = 8, kPer = 2 * kRun, kHalf = kRun / 2;

enum { kToTensors = 0, kToBf16 = 1, kToF8 = 2 };
enum { kNoTurn = 0, kNeighbours = 1, kHalves = 2, kRaggedHalves = 3 };

// Eight elements of T as they lie in memory.
template <typename T>
struct Run {
  static constexpr int kPieces = (int)sizeof(T) / 2;
  uint32_t w[4 * kPieces];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
};

// A run as pairs of floats, and back
__device__ __forceinline__ void widen(const Run<__nv_bfloat16>& r, unsigned long long* p) {
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i)
    p[i] = pair(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
}
__device__ __forceinline__ void widen(const Run<float>& r, unsigned long long* p) {
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i)
    p[i] = pair(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
}
__device__ __forceinline__ void put(__nv_bfloat16* to, const unsigned long long* p) {
  Run<__nv_bfloat16> r;
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) {
    float x, y;
    unpair(p[i], &x, &y);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  r.store(to);
}
__device__ __forceinline__ void put(float* to, const unsigned long long* p) {
  Run<float> r;
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) {
    float x, y;
    unpair(p[i], &x, &y);
    r.w[2 * i] = __float_as_uint(x), r.w[2 * i + 1] = __float_as_uint(y);
  }
  r.store(to);
}

// Heads of one kind of one token: what a lane group works on at a time.
template <typename T>
struct Unit {
  const T* src;                            // this lane's first run of the first head
  long long stride;                        // between heads
  int count;                               // heads; 0: none
  int kind;                                // 0 queries, 1 keys, 2 values
  int head, t;                             // the first head, the token of the group
};

// Four floats a lane, piece by piece: what lane l wants of a row of L kPer elements in pieces of
// four lies at [piece][l], so that lanes read it side by side.
template <int L>
__device__ __forceinline__ int place(int lane, int e) { return (e / 4 * L + lane) * 4 + e % 4; }

// Grid: x groups of a.tokens (<= kTokens) tokens, y parts of a token group's units.  L: a power of
// two, D <= kPer L.
template <typename T, int L, int kTo, int kTokens, int kHeads, bool kRagged>
__global__ void __launch_bounds__(kThreads, kRagged ? 4 : 6) gdn_qk_norm_rope_kernel(GdnRopeArgs a) {
  constexpr int kGroups = kThreads / L;
  pdl_wait();                              // (nothing is read before)
  __shared__ float4 s_cos[kTokens][kRun / 4][L], s_sin[kTokens][kRun / 4][L];   // of a lane's pairs
  __shared__ float4 s_weight[2][kPer / 4][L];
  __shared__ long long s_row[kTokens];     // of head 0 of the token's slot (-1: none)
  // ragged halves: cos and sin (negative for the first half) of each element, a vector a lane group
  extern __shared__ float4 s_ragged[];
  constexpr int kRow = kPer / 4 * L;
  float4* const s_of = s_ragged;           // [token][cos, sin][kRow]
  float* const s_stage = reinterpret_cast<float*>(s_ragged + kTokens * 2 * kRow) +
                         threadIdx.x / L * (L * kPer);
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  // the lanes of this group, whose branches are the same
  const uint32_t peers = (0xffffffffu >> (32 - L)) << (threadIdx.x % 32 / L * L);
  const int D = a.D, r = a.rotary;
  const int t0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.n - t0);
  // this lane's runs, the second `gap` elements behind the first
  const bool halves = !kRagged && a.turn == kHalves;
  auto first_of = [&](int l) { return halves && l * kPer < r ? l * kRun : l * kPer; };
  auto gap_of = [&](int l) { return halves && l * kPer < r ? r / 2 : kRun; };
  const int e0 = first_of(lane), gap = gap_of(lane);
  const bool turns = lane * kPer < r && !kRagged;
  const bool mine = e0 < D, both = e0 + gap < D;       // (D is a multiple of eight)
  const int units_q = (a.Hq + kHeads - 1) / kHeads, units_h = (a.H + kHeads - 1) / kHeads;
  const int per = units_q + units_h * (kTo == kToTensors ? 1 : 2), all = tokens * per;
  const int step = kGroups * gridDim.y;
  auto unit_of = [&](int i) {
    Unit<T> u;
    u.t = 0;
#pragma unroll
    for (int k = 1; k < kTokens; ++k) u.t += i >= k * per ? 1 : 0;
    int j = i - u.t * per;
    u.kind = j < units_q ? 0 : j < units_q + units_h ? 1 : 2;
    j -= u.kind == 0 ? 0 : u.kind == 1 ? units_q : units_q + units_h;
    u.head = j * kHeads;
    u.count = i < all ? min(kHeads, (u.kind == 0 ? a.Hq : a.H) - u.head) : 0;
    const long long tok = t0 + u.t;
    u.stride = u.kind == 0 ? a.q_head : D;
    u.src = (u.kind == 0   ? (const T*)a.q + tok * a.q_tok
             : u.kind == 1 ? (const T*)a.k + tok * a.k_tok
                           : (const T*)a.v + tok * a.v_tok) + u.head * u.stride + e0;
    if (!in_bounds(&g_err_kv, u.count <= 0 || tok < a.n)) u.count = 0;
    return u;
  };
  Run<T> raw[kHeads][2];
  auto load = [&](const Unit<T>& u, int v) {
    if (v >= u.count || !mine || !in_bounds(&g_err_kv, e0 + kRun <= D)) return;
    raw[v][0].load(u.src + v * u.stride);
    if (both && in_bounds(&g_err_kv, e0 + gap + kRun <= D)) raw[v][1].load(u.src + v * u.stride + gap);
  };
  int i0 = blockIdx.y * kGroups + group;
  Unit<T> u = unit_of(i0);
#pragma unroll
  for (int v = 0; v < kHeads; ++v) load(u, v);
  // ---- cos and sin of the tokens' angles, the weights, the tokens' places in the cache
  for (int i = threadIdx.x; i < tokens * (r / 2); i += kThreads) {
    const int t = i / (r / 2), p = i - t * (r / 2);
    if (!in_bounds(&g_err_kv, t0 + t < a.n && p < kMaxPairs)) break;
    const uint64_t phase = (uint64_t)(int64_t)a.positions[t0 + t] * a.steps[p];
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
    cs *= a.amplitude, sn *= a.amplitude;
    if (!kRagged) {
      reinterpret_cast<float*>(s_cos[t])[place<L>(p / kRun, p % kRun)] = cs;
      reinterpret_cast<float*>(s_sin[t])[place<L>(p / kRun, p % kRun)] = sn;
      continue;
    }
    float* of = reinterpret_cast<float*>(s_of + t * 2 * kRow);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = p + h * (r / 2), at = place<L>(e / kPer, e % kPer);
      of[at] = cs;
      of[4 * kRow + at] = h ? sn : -sn;
    }
  }
  if (kRagged) {                           // the elements behind the turned ones
    for (int i = threadIdx.x; i < tokens * (L * kPer - r); i += kThreads) {
      const int t = i / (L * kPer - r), e = r + i - t * (L * kPer - r);
      float* of = reinterpret_cast<float*>(s_of + t * 2 * kRow);
      of[place<L>(e / kPer, e % kPer)] = 1.0f;
      of[4 * kRow + place<L>(e / kPer, e % kPer)] = 0.0f;
    }
  }
  for (int i = threadIdx.x; i < 2 * (kPer / 4) * L; i += kThreads) {
    const int l = i % L, k = i / L % (kPer / 4), kind = i / (L * (kPer / 4));
    const float* w = kind ? a.wk : a.wq;
    const int e = first_of(l) + (k < kRun / 4 ? 0 : gap_of(l) - kRun) + k * 4;
    if (w && e < D) s_weight[kind][k][l] = *reinterpret_cast<const float4*>(w + e);
  }
  if (kTo != kToTensors && (int)threadIdx.x < tokens)
    s_row[threadIdx.x] = kv_row_of(&g_err_kv, a.cache, a.slots[t0 + threadIdx.x], 0);
  __syncthreads();

  for (; i0 - group < all; i0 += step) {   // (the same for all groups of a block)
    const Unit<T> next = unit_of(i0 + step);
    const bool norm = u.kind == 0 ? a.wq != nullptr : u.kind == 1 && a.wk != nullptr;
    const bool turn = turns && u.kind < 2 && u.count > 0;
    // where this lane's runs of the first head go
    const long long tok = t0 + u.t;
    T* out = u.kind == 0 ? (T*)a.q_out + tok * a.q_out_tok + (long long)u.head * D + e0
             : u.kind == 1 && a.k_out ? (T*)a.k_out + (tok * a.H + u.head) * D + e0
                                      : nullptr;
    long long row = -1;                    // of the cache
    if (kTo != kToTensors && u.kind > 0 && u.count > 0 && s_row[u.t] >= 0)
      row = s_row[u.t] + ((long long)u.head << a.cache.page_shift);
#pragma unroll
    for (int v = 0; v < kHeads; ++v) {
      const bool live = v < u.count && mine;
      unsigned long long p[kRun];          // pairs of elements: the first run's, the second's
      widen(raw[v][0], p);
      widen(raw[v][1], p + kHalf);
      if (!both)
#pragma unroll
        for (int k = 0; k < kHalf; ++k) p[kHalf + k] = 0;
      load(next, v);
      // ---- the norm (lanes without elements hold nothing)
      if (norm) {
        unsigned long long sum2 = mul2(p[0], p[0]);
#pragma unroll
        for (int k = 1; k < kRun; ++k) sum2 = fma2(p[k], p[k], sum2);
        float s0, s1;
        unpair(sum2, &s0, &s1);
        float sum = live ? s0 + s1 : 0.0f;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(peers, sum, o);
        const float f = rsqrtf(sum * a.inv_d + a.eps);
        const unsigned long long f2 = pair(f, f);
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) {
          const float4 w = s_weight[u.kind][k][lane];
          p[2 * k] = mul2(p[2 * k], mul2(pair(w.x, w.y), f2));
          p[2 * k + 1] = mul2(p[2 * k + 1], mul2(pair(w.z, w.w), f2));
        }
      }
      // ---- the rotation
      if (turn) {
        unsigned long long cs[kHalf], sn[kHalf];
#pragma unroll
        for (int k = 0; k < kRun / 4; ++k) {
          const float4 c = s_cos[u.t][k][lane], s = s_sin[u.t][k][lane];
          cs[2 * k] = pair(c.x, c.y), cs[2 * k + 1] = pair(c.z, c.w);
          sn[2 * k] = pair(s.x, s.y), sn[2 * k + 1] = pair(s.z, s.w);
        }
        if (halves) {
#pragma unroll
          for (int k = 0; k < kHalf; ++k) {
            const unsigned long long lo = p[k], hi = p[k + kHalf];
            float s0, s1;
            unpair(sn[k], &s0, &s1);
            p[k] = fma2(lo, cs[k], mul2(hi, pair(-s0, -s1)));
            p[k + kHalf] = fma2(hi, cs[k], mul2(lo, sn[k]));
          }
        } else {
#pragma unroll
          for (int k = 0; k < kRun; ++k) {
            float x0, x1, c[2], s[2];
            unpair(p[k], &x0, &x1);
            unpair(cs[k / 2], &c[0], &c[1]);
            unpair(sn[k / 2], &s[0], &s[1]);
            if (lane * kPer + 2 * k < r)
              p[k] = pair(x0 * c[k & 1] - x1 * s[k & 1], x0 * s[k & 1] + x1 * c[k & 1]);
          }
        }
      }
      if constexpr (kRagged) {
        float y[kPer];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) {
          unpair(p[2 * k], &y[4 * k], &y[4 * k + 1]);
          unpair(p[2 * k + 1], &y[4 * k + 2], &y[4 * k + 3]);
          reinterpret_cast<float4*>(s_stage)[k * L + lane] =
              make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        }
        __syncwarp();
        if (u.kind < 2) {
          const float4* of = s_of + u.t * 2 * kRow;
#pragma unroll
          for (int k = 0; k < kPer / 4; ++k) {
            const float4 c4 = of[k * L + lane], s4 = of[kRow + k * L + lane];
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = lane * kPer + 4 * k + e;
              const int other = at < r / 2 ? at + r / 2 : at < r ? at - r / 2 : at;
              const float z = s_stage[place<L>(other / kPer, other % kPer)];
              const float turned = y[4 * k + e] * c[e] + z * sn[e];
              y[4 * k + e] = at < r ? turned : y[4 * k + e];
            }
          }
#pragma unroll
          for (int k = 0; k < kRun; ++k) p[k] = pair(y[2 * k], y[2 * k + 1]);
        }
      }
      // ---- out
      if (live && out && in_bounds(&g_err_kv, tok < a.n && e0 + kRun <= D)) {
        put(out + v * D, p);
        if (both && in_bounds(&g_err_kv, e0 + gap + kRun <= D)) put(out + v * D + gap, p + kHalf);
      }
      if constexpr (kTo == kToBf16) {
        if (live && row >= 0 && in_bounds(&g_err_kv, u.head + v < a.H && e0 + gap + kRun <= D)) {
          __nv_bfloat16* to = (__nv_bfloat16*)(u.kind == 2 ? a.cache.v : a.cache.k) +
                              (row + ((long long)v << a.cache.page_shift)) * D + e0;
          put(to, p);
          put(to + gap, p + kHalf);
        }
      }
      if constexpr (kTo == kToF8) {
        if (u.kind > 0) {
          float y[kPer], top = 0.0f;
#pragma unroll
          for (int k = 0; k < kRun; ++k) unpair(p[k], &y[2 * k], &y[2 * k + 1]);
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const float m = fabsf(y[k]);
            top = m < INFINITY ? fmaxf(top, m) : top;
          }
          top = live ? top : 0.0f;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(peers, top, o));
          const int e = kv_scale_exponent(top);
          if (live && row >= 0 && in_bounds(&g_err_kv, u.head + v < a.H && e0 + gap + kRun <= D)) {
            const long long at = row + ((long long)v << a.cache.page_shift);
            uint8_t* to = (uint8_t*)(u.kind == 2 ? a.cache.v : a.cache.k) + at * D + e0;
            *reinterpret_cast<uint2*>(to) = make_uint2(kv_codes4(y, e), kv_codes4(y + 4, e));
            *reinterpret_cast<uint2*>(to + gap) =
                make_uint2(kv_codes4(y + 8, e), kv_codes4(y + 12, e));
            if (lane == 0) (u.kind == 2 ? a.cache.v_exp : a.cache.k_exp)[at] = (uint8_t)(e + 127);
          }
        }
      }
    }
    u = next;
  }
  // Only now: CTAs of the next kernel that came earlier would land where this one leaves room,
  // unevenly (2501 tokens in fp32 13.1 us, so 11.9; with an ordinary launch 14.4 in a stream).
  pdl_trigger();
}

template <typename T, int L, int kTo, int kTokens, int kHeads, bool kRagged>
cudaError_t launch(GdnRopeArgs a, int tokens, int parts, cudaStream_t stream) {
  const size_t smem = kRagged ? sizeof(float) * kPer * (kTokens * 2 * L + kThreads) : 0;
  a.tokens = tokens;
  const dim3 grid((unsigned)((a.n + (long long)tokens - 1) / tokens), (unsigned)parts);
  // (set up while the kernel before ends: 128 tokens into the 8-bit cache 6.2 -> 3.9 us in a stream)
  return launch_pdl(true, gdn_qk_norm_rope_kernel<T, L, kTo, kTokens, kHeads, kRagged>, grid,
                    dim3(kThreads), smem, stream, a);
}

template <typename T, int L, int kTo>
cudaError_t launch(const GdnRopeArgs& a, cudaStream_t stream) {
  constexpr int kGroups = kThreads / L;
  const int per = a.Hq + a.H * (kTo == kToTensors ? 1 : 2);
  // Tokens of a CTA, which share the cost of its start: as few as let all CTAs run at once (six an
  // SM).  24 + 4 + 4 heads of 256 in bf16, one, two, three and four a CTA: 600 tokens 5.9 / 7.3 / - / 10.4
  // us, 1200 12.1 / 11.1 / - / 13.6, 2500 19.8 / 19.9 / 17.7 / 19.4; 4 + 4 + 4: 3000 14.0 / 11.4 / 12.3 /
  // 9.0; 16 + 2 of 128 in fp32: 1200 8.4 / 6.8 / - / 6.8, 2500 14.4 / 14.7 / 12.4 / 12.9, 10000 43.8 / 40.3 /
  // - / 37.3.  (Up to eight cost the others: 16384 tokens 89 us, so 97 to 105.)
  const int tokens = (int)std::min(4ll, (a.n + 152ll * 6 - 1) / (152 * 6));
  // Few vectors: one a lane group, so that all of them are on the way at once.
  const bool few = (long long)a.n * per <= 152ll * 4 * kGroups;
  const int parts = few ? (per + kGroups - 1) / kGroups : 1;
  if (a.turn == kRaggedHalves) return launch<T, L, kTo, 4, 1, true>(a, few ? 1 : tokens, parts, stream);
  if (few) return launch<T, L, kTo, 1, 1, false>(a, 1, parts, stream);
  // Heads at a time: two of bf16 (registers; the large case of one 94 us, two 89, four 96), one of
  // fp32 (two spill: 15.4 us where one takes 13.0).
  return launch<T, L, kTo, 4, sizeof(T) == 2 ? 2 : 1, false>(a, tokens, 1, stream);
}

template <typename T, int L>
cudaError_t launch(const GdnRopeArgs& a, cudaStream_t stream) {
  if constexpr (kPer * L >= 128) {         // a cache's heads have 128 or 256 elements
    if (a.to_cache && a.cache.f8) return launch<T, L, kToF8>(a, stream);
    if (a.to_cache) return launch<T, L, kToBf16>(a, stream);
  }
  return launch<T, L, kToTensors>(a, stream);
}

template <typename T>
cudaError_t launch(const GdnRopeArgs& a, cudaStream_t stream) {
  if (a.D > 128) return launch<T, 16>(a, stream);
  if (a.D > 64) return launch<T, 8>(a, stream);
  return launch<T, 4>(a, stream);
}

}  // namespace rope
}  // namespace

cudaError_t gdn_launch_qk_norm_rope(GdnRopeArgs a, int in_bf16, cudaStream_t stream) {
  a.inv_d = 1.0f / (float)a.D;
  a.turn = a.rotary == 0 ? rope::kNoTurn
           : a.interleaved ? rope::kNeighbours
           : a.rotary % rope::kPer == 0 ? rope::kHalves
                                        : rope::kRaggedHalves;
  return in_bf16 ? rope::launch<__nv_bfloat16>(a, stream) : rope::launch<float>(a, stream);
}
