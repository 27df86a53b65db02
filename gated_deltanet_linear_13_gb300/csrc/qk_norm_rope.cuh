// The norm of query and key heads with their rotation by position, and the write of keys and
// values to the paged cache, in one pass.
//
// Per head vector x of D elements: y = x rsqrt(mean x^2 + eps) w, then each pair (a, b) of its
// first r elements is turned by the angle w_p = position * frequency_p.  The angle is kept as a
// phase in 2^64ths of a turn: position * step_p modulo 2^64 is one 64-bit product, exact for every
// position (in 32 bits an angle of 10^6 radians is off by 0.03), and its upper 32 bits give cos and
// sin to 2^-31 of a turn.  All in fp32, rounded once to what is stored; an 8-bit cache is
// quantised from the fp32 keys.
//
// D / 8 lanes a vector, eight elements a lane, so a pair's halves lie in one lane (interleaved), in
// lanes rotary_dim / 16 apart (halves, where rotary_dim / 2 is a multiple of eight: a shuffle), or
// go through shared memory.  A token's cos and sin are made once for all its heads.
// Part of kv_cache.cu, whose error word it uses.
#pragma once

#include "common.cuh"
#include "kv_cache.cuh"

using namespace gdn;

namespace {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

enum { kToTensors = 0, kToBf16 = 1, kToF8 = 2 };
enum { kNoTurn = 0, kNeighbours = 1, kHalvesShuffled = 2, kHalves = 3 };

// Grid: x groups of kTokens tokens, y parts of the vectors of a token group.  L lanes a vector
// (a power of two, D <= 8 L), `kAhead` vectors of a group on the way at a time.
template <typename T, int L, int kTo, int kTokens, int kAhead>
__global__ void __launch_bounds__(kThreads) gdn_qk_norm_rope_kernel(GdnRopeArgs a) {
  constexpr int kGroups = kThreads / L;
  __shared__ __align__(16) float2 s_turn[kTokens][kMaxPairs];
  __shared__ __align__(16) float s_stage[kThreads / 32][256];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int D = a.D, r = a.rotary, e0 = lane * 8;
  const int t0 = blockIdx.x * kTokens, tokens = min(kTokens, a.n - t0);
  const bool mine = e0 < D;
  // queries, keys, and with a cache the values
  const int per = a.Hq + a.H * (kTo == kToTensors ? 1 : 2), all = tokens * per;
  // ---- cos and sin of the tokens' angles
  for (int i = threadIdx.x; i < tokens * (r / 2); i += kThreads) {
    const int t = i / (r / 2), p = i - t * (r / 2);
    if (!in_bounds(&g_err_kv, t0 + t < a.n && p < kMaxPairs)) break;
    const uint64_t phase = (uint64_t)(int64_t)a.positions[t0 + t] * a.steps[p];
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
    s_turn[t][p] = make_float2(cs * a.amplitude, sn * a.amplitude);
  }
  Vec8 wq, wk;
#pragma unroll
  for (int e = 0; e < 8; ++e) wq.x[e] = wk.x[e] = 1.0f;
  if (a.wq && mine) wq = load8(a.wq + e0);
  if (a.wk && mine) wk = load8(a.wk + e0);
  __syncthreads();

  const int step = kGroups * gridDim.y;
  for (int i0 = blockIdx.y * kGroups + group; i0 - group < all; i0 += step * kAhead) {
    Vec8 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * step;
      x[u] = Vec8{};
      if (i < all && mine) {
        const int t = i / per, h = i - t * per;
        const long long tok = t0 + t;
        const T* src = h < a.Hq ? (const T*)a.q + tok * a.q_tok + h * a.q_head
                       : h < a.Hq + a.H
                           ? (const T*)a.k + tok * a.k_tok + (long long)(h - a.Hq) * D
                           : (const T*)a.v + tok * a.v_tok + (long long)(h - a.Hq - a.H) * D;
        if (in_bounds(&g_err_kv, tok < a.n)) x[u] = load8(src + e0);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * step;
      const int t = min(i, all - 1) / per, h = min(i, all - 1) - t * per;
      const long long tok = t0 + t;
      const bool query = h < a.Hq, value = h >= a.Hq + a.H;
      Vec8 y = x[u];
      // ---- the norm
      const float* w = query ? a.wq : a.wk;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(y.x[e], y.x[e], sum);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (w && !value) {
        const float f = rsqrtf(sum * a.inv_d + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) y.x[e] *= f * (query ? wq.x[e] : wk.x[e]);
      }
      // ---- the rotation
      if (a.turn == kNeighbours) {
        if (e0 < r && !value) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            if (e0 + 2 * p >= r) continue;
            const float2 c = s_turn[t][e0 / 2 + p];
            const float u0 = y.x[2 * p], u1 = y.x[2 * p + 1];
            y.x[2 * p] = u0 * c.x - u1 * c.y;
            y.x[2 * p + 1] = u0 * c.y + u1 * c.x;
          }
        }
      } else if (a.turn == kHalvesShuffled) {
        const int half = r / 2, off = half / 8;
        const bool low = e0 < half;
        const int from = (threadIdx.x & 31) + (low ? off : -off);
        Vec8 z;
#pragma unroll
        for (int e = 0; e < 8; ++e) z.x[e] = __shfl_sync(0xffffffffu, y.x[e], from & 31);
        if (e0 < r && !value) {
          const float2* c = &s_turn[t][low ? e0 : e0 - half];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y.x[e] = y.x[e] * c[e].x + (low ? -z.x[e] : z.x[e]) * c[e].y;
        }
      } else if (a.turn == kHalves) {
        float* row = &s_stage[threadIdx.x / 32][((threadIdx.x & 31) / L) * (L * 8)];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) row[e0 + e] = y.x[e];
        __syncwarp();
        if (!value) {
          const int half = r / 2;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = e0 + e;
            if (at >= r) continue;
            const bool low = at < half;
            const float2 c = s_turn[t][low ? at : at - half];
            const float z = row[low ? at + half : at - half];
            y.x[e] = y.x[e] * c.x + (low ? -z : z) * c.y;
          }
        }
      }
      // ---- out
      const bool live = i < all && mine && in_bounds(&g_err_kv, tok < a.n && e0 + 8 <= D);
      if (query) {
        if (live) store8((T*)a.q_out + tok * a.q_out_tok + (long long)h * D + e0, y);
      }
      if (!query && a.k_out && !value && live)
        store8((T*)a.k_out + (tok * a.H + (h - a.Hq)) * D + e0, y);
      if constexpr (kTo != kToTensors) {
        const int head = query ? 0 : h - a.Hq - (value ? a.H : 0);
        long long row = -1;
        if (!query && i < all) row = kv_row_of(&g_err_kv, a.cache, a.slots[tok], head);
        if constexpr (kTo == kToBf16) {
          if (row >= 0 && live)
            store8((__nv_bfloat16*)(value ? a.cache.v : a.cache.k) + row * D + e0, y);
        } else {
          float top = kv_largest(y);
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = kv_scale_exponent(top);
          if (row >= 0 && live) {
            *reinterpret_cast<uint2*>((uint8_t*)(value ? a.cache.v : a.cache.k) + row * D + e0) =
                kv_codes(y, e);
            if (lane == 0) (value ? a.cache.v_exp : a.cache.k_exp)[row] = (uint8_t)(e + 127);
          }
        }
      }
    }
  }
}

template <typename T, int L, int kTo>
cudaError_t launch(const GdnRopeArgs& a, cudaStream_t stream) {
  constexpr int kGroups = kThreads / L;
  const int per = a.Hq + a.H * (kTo == kToTensors ? 1 : 2);
  // Few vectors: one a group of lanes, so that all of them are on the way at once.
  if ((long long)a.n * per <= 152ll * 8 * kGroups) {
    const dim3 grid((unsigned)a.n, (unsigned)((per + kGroups - 1) / kGroups));
    gdn_qk_norm_rope_kernel<T, L, kTo, 1, 1><<<grid, kThreads, 0, stream>>>(a);
  } else {
    constexpr int kTokens = 4;
    const dim3 grid((unsigned)((a.n + kTokens - 1) / kTokens), 1);
    gdn_qk_norm_rope_kernel<T, L, kTo, kTokens, 4><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, int L>
cudaError_t launch(const GdnRopeArgs& a, cudaStream_t stream) {
  if constexpr (L >= 16) {                 // a cache's heads have 128 or 256 elements
    if (a.to_cache && a.cache.f8) return launch<T, L, kToF8>(a, stream);
    if (a.to_cache) return launch<T, L, kToBf16>(a, stream);
  }
  return launch<T, L, kToTensors>(a, stream);
}

template <typename T>
cudaError_t launch(const GdnRopeArgs& a, cudaStream_t stream) {
  if (a.D > 128) return launch<T, 32>(a, stream);
  if (a.D > 64) return launch<T, 16>(a, stream);
  return launch<T, 8>(a, stream);
}

}  // namespace rope
}  // namespace

cudaError_t gdn_launch_qk_norm_rope(GdnRopeArgs a, int in_bf16, cudaStream_t stream) {
  a.inv_d = 1.0f / (float)a.D;
  a.turn = a.rotary == 0 ? rope::kNoTurn
           : a.interleaved ? rope::kNeighbours
           : a.rotary % 16 == 0 ? rope::kHalvesShuffled
                                : rope::kHalves;
  return in_bf16 ? rope::launch<__nv_bfloat16>(a, stream) : rope::launch<float>(a, stream);
}
