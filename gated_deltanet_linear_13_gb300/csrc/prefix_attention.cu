// Attention of a batch that shares a long prefix, over the paged key/value cache.
//
// Work.  The rows (token, query head) that read the same keys form a unit: the rows of the whole
// batch for one key/value head of the prefix, the rows of one sequence for one key/value head of
// its own tokens, each cut into row tiles of 128.  A unit's keys are cut into tiles of 128.  All
// (unit, key tile) pairs lie on one line, units one after the other; CTA c of the grid takes the
// c-th equal part of it (a unit's start counts as some tiles too), so that every SM streams the
// same number of keys whatever the lengths.  A unit's parts leave unnormalised outputs with each
// row's reference m and sum l; the merge kernel joins a row's parts, prefix and own alike:
//     out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.
// The line is laid out on the device from the lengths, so a captured call can be replayed as they
// grow.
//
// A part: S = Q K^T (M = 128 rows, N = 128 keys) and O += P V on tcgen05, S double-buffered in
// tensor memory, P written over its S and read from there as the A operand; a running reference
// m per row (raised, with O rescaled, only when the maximum passes it by more than kSlack, so
// that a rescale is rare; any reference is exact, it cancels).  Two producer warps stream K and V
// tiles by TMA through a ring in shared memory, one copy a page (one warp: 3.1 us a tile of
// 16-token pages, two: 2.4).  P takes two bf16 terms, the leading bits and the rounded rest, so
// that the output is as exact as fp32 sums make it: half of the second product's time again.
//
// 8-bit cache: the codes are the operands as they lie in memory, nothing is converted on the way
// to the tensor cores.  A bf16 element of Q, scaled by a power of two per row, is the sum of two
// e4m3 numbers (4 + 4 significant bits; only elements below 2^-10 of the row's largest lose
// bits), so S is two 8-bit products at twice the bf16 rate.  P takes three e5m2 terms (3 bits
// each and the terms' signs: 11 bits; e5m2 for its range: the smallest probabilities matter when
// a few keys outweigh thousands).  The keys' scales multiply the scores; the values' scales 2^e_j
// go into the exponent, P'_j = 2^(t_j + e_j - m) with m bounding t_j + e_j, and come out of the row
// sum again, l = sum_j P'_j 2^(-e_j).
//
// Large scores.  t - m in one rounding, s c - m, holds as long as m = fl(max c) rounds by little
// (kNear, common.cuh).  With a bf16 cache a row beyond that takes (s - max) c, and its parts are
// joined by the scores that their references are of.  With an 8-bit cache t + e_j is rounded as a
// score of its own, and a large maximum is its own reference.
//
// Bound: many keys a row tile by the products (D = 256: 2.25 us a tile of 128 keys in bf16, 1.6 in
// 8 bits: over the three and the five products 87% of the bf16 rate of a library matrix product
// and about twice that rate; D = 128: 1.2 us, the chain score, softmax, product); many short
// sequences by memory (128 sequences of up to 2048 tokens of their own on 4096: 104 us, 5.0 TB/s);
// a few keys by latency (one request on 512 + 37 keys: 12 us with the merge).  Measured in whole:
// 32 sequences on 16384, 8-bit, 43 us; 16 x 4 tokens on 32771, bf16, 73; 666 tokens on 20000,
// D = 128, 127.
#include <float.h>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

using namespace gdn;
using namespace gdn::ptx;

static __device__ unsigned int g_err_attn;

unsigned gdn_take_error_prefix_attention() { return gdn::take_error(g_err_attn); }

namespace {

constexpr int kCtas = 152;                 // one CTA an SM
constexpr int kRows = 128, kKeys = 128;
// Rows of all heads up to which the merge's warps share out a row's parts (shared / not, in whole:
// 32 sequences of 24 heads 39.5 / 43.9 us, 64: 61.6 / 62.6, 100: 92.5 / 91.1, 128: 107.8 / 103.6).
constexpr int kFewRows = 2048;
constexpr long long kBlockBytes = 256ll << 20;
// parts whose reference m lies past it leave the score that m is of as well
constexpr float kFar = 0.25f * kNear;
constexpr int KB = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Warps: 0, 3 producers, 1 MMA issuer, 2 the 8-bit cache's scales, 4-11 softmax (two a TMEM lane
// quarter, 64 of the tile's keys each).
constexpr int kThreads = 384, kSoftmaxWarps = 8;

template <int D, bool kF8>
struct Shape {
  static constexpr int kSlotBytes = kF8 ? kKeys * D : kKeys * 256;   // keys x at most 256 bytes
  static constexpr int kSlotsPerTile = kF8 ? 1 : D / 128;           // of K, and of V
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kSlots = kF8 ? (D == 256 ? 4 : 8) : (D == 256 ? 5 : 6);
  static constexpr int kElem = kF8 ? 128 : 64;                       // elements of a 128-byte row
  // shared memory
  static constexpr int kRing = kQBytes;
  static constexpr int kMax = kRing + kSlots * kSlotBytes;           // [2][2][128] float
  static constexpr int kSum = kMax + 2048;                           // [128] float
  static constexpr int kQFac = kSum + 512;                           // [2][128] float (8-bit)
  static constexpr int kScales = kQFac + (kF8 ? 1024 : 0);            // [2][3][128] float (8-bit)
  static constexpr int kBars = kScales + (kF8 ? 3072 : 0);
  static constexpr int kMisc = kBars + 8 * (2 * kSlots + 12 + 1);
  static constexpr int kBytes = kMisc + 64;
};
static_assert(Shape<256, false>::kBytes <= 227 * KB && Shape<256, true>::kBytes <= 227 * KB &&
                  Shape<128, false>::kBytes <= 227 * KB && Shape<128, true>::kBytes <= 227 * KB,
              "shared memory");

// tensor memory (columns)
constexpr uint32_t TM_S = 0, TM_O = 256;

struct Params {
  GdnAttnArgs a;
  int G, row_tiles_p, row_tiles_s, prefix_tiles;
  int unit_cost;                   // tiles that a unit's start and end are worth
  float coef;                      // see score_unit
  int blocks, block_tiles;         // the prefix's key tiles, cut into blocks (the last shorter)
  int rows_p, rows_s;              // rows stored a part (<= 128)
  float *o_p, *o_s;                // parts: [slot][D / 4][rows][4]
  float2 *ml_p, *ml_s;             // [slot][rows]: m (base 2), l
  float *far_p, *far_s;            // [slot][rows]: where |m| > kFar, the score m is of (bf16 cache)
  int2 *span_p, *span_s;           // [unit]: the CTAs that have its first and its last tile
};

__device__ __forceinline__ int own_len(const GdnAttnArgs& a, int b) {
  const int n = a.kv_len[b], most = a.max_pages << a.cache.page_shift;
  return n > most ? most : n;
}
// keys that some row of row tile rt of a sequence of n tokens sees (the last row's)
__device__ __forceinline__ int tile_keys(const Params& p, int n, int rt) {
  const int last = (rt + 1) * kRows - 1;              // (of the last tile: no division)
  const int t = rt + 1 == p.row_tiles_s ? p.a.T - 1 : last / p.G;
  return max(0, min(n, n - p.a.T + 1 + t));
}
__device__ __forceinline__ int key_tiles(int keys) { return (keys + kKeys - 1) / kKeys; }
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
// a unit's length on the line
__device__ __forceinline__ int unit_len(const Params& p, int tiles) {
  return tiles > 0 ? tiles + p.unit_cost : 0;
}
__device__ __forceinline__ long long seq_len_on_line(const Params& p, int b) {
  const int n = own_len(p.a, b);
  long long w = 0;
  if (n > 0)
    for (int rt = 0; rt < p.row_tiles_s; ++rt) w += unit_len(p, key_tiles(tile_keys(p, n, rt)));
  return w * p.a.cache.H;
}

// The prefix's units lie in the order (head, block of keys, row tile): the row tiles of a block
// side by side, so that the CTAs that read the same keys do so at the same time, out of L2.
__device__ __forceinline__ int block_len(const Params& p, int blk) {
  return unit_len(p, min(p.block_tiles, p.prefix_tiles - blk * p.block_tiles));
}
__device__ __forceinline__ long long head_len(const Params& p) {
  if (p.prefix_tiles == 0) return 0;
  return (long long)p.row_tiles_p *
         ((long long)(p.blocks - 1) * unit_len(p, p.block_tiles) + block_len(p, p.blocks - 1));
}

// What the workspace has room for (index checks): units, and parts' slots.
__device__ __forceinline__ long long unit_room(const Params& p, bool prefix) {
  return prefix ? max((long long)p.a.cache.H * p.row_tiles_p, (long long)kCtas)
                : (long long)p.a.B * p.row_tiles_s * p.a.cache.H;
}
__device__ __forceinline__ bool in_workspace(const Params& p, bool prefix, long long unit, int c,
                                             int r) {
  return in_bounds(&g_err_attn, unit >= 0 && unit < unit_room(p, prefix) && c >= 0 && c < kCtas &&
                                    r >= 0 && r < (prefix ? p.rows_p : p.rows_s));
}

// One CTA's piece of a unit.
struct Item {
  bool prefix, first, last; // the prefix's or a sequence's; has the unit's first, last tile
  int h, b, rt, n;          // head, sequence, row tile, the sequence's own tokens
  int keys, j0, j1;         // keys some row sees; key tiles [j0, j1)
  long long unit;           // index among the prefix's / the sequences' units
};

// Walks the pieces of [pos, end) of the line; the same sequence in every warp.
struct Walk {
  long long pos, end, at;   // at: where the current unit starts
  bool prefix;
  int b, blk, rt, h;
  int n, keys, tiles;       // the current unit's sequence length, keys and key tiles

  // for the unit at (b, rt), which changed
  __device__ __forceinline__ void measure(const Params& p, bool other_sequence) {
    if (prefix) {
      n = 0;
      keys = p.a.prefix_len;
      tiles = min(p.block_tiles, p.prefix_tiles - blk * p.block_tiles);
      return;
    }
    if (b >= p.a.B) return;
    if (other_sequence) n = own_len(p.a, b);
    keys = n > 0 ? tile_keys(p, n, rt) : 0;
    tiles = key_tiles(keys);
  }

  __device__ void start(const Params& p, long long lo, long long hi, int b0, long long at0) {
    pos = lo; end = hi;
    const long long hl = head_len(p);
    prefix = lo < hl * p.a.cache.H;
    b = prefix ? 0 : b0; blk = 0; rt = 0; h = 0;
    at = at0;
    if (prefix) {
      h = (int)quotient(lo, hl);
      long long rest = lo - h * hl;
      const long long bl = (long long)p.row_tiles_p * unit_len(p, p.block_tiles);
      blk = min((int)quotient(rest, bl), p.blocks - 1);
      rest -= blk * bl;
      rt = (int)quotient(rest, block_len(p, blk));
      at = h * hl + blk * bl + (long long)rt * block_len(p, blk);
    }
    measure(p, true);
    if (!prefix && b < p.a.B && lo < hi) {
      // the units of the sequence before lo
      while (lo - at >= (long long)p.a.cache.H * unit_len(p, tiles) && rt + 1 < p.row_tiles_s) {
        at += (long long)p.a.cache.H * unit_len(p, tiles);
        ++rt;
        measure(p, false);
      }
      if (tiles > 0) h = (int)quotient(lo - at, unit_len(p, tiles));
      at += (long long)h * unit_len(p, tiles);
    }
  }
  __device__ bool next(const Params& p, Item* it) {
    const int H = p.a.cache.H;
    while (at < end) {
      int base = 0;
      if (prefix) {
        base = blk * p.block_tiles;
        it->unit = ((long long)h * p.blocks + blk) * p.row_tiles_p + rt;
      } else {
        if (b >= p.a.B) return false;
        it->unit = ((long long)b * p.row_tiles_s + rt) * H + h;
      }
      it->prefix = prefix;
      it->keys = keys; it->n = n;
      it->h = h; it->rt = rt; it->b = b;
      const long long first = at + p.unit_cost;
      const long long j0 = pos > first ? pos - first : 0;
      const long long j1 = end > first ? end - first : 0;
      it->j0 = base + (int)(j0 < tiles ? j0 : tiles);
      it->j1 = base + (int)(j1 < tiles ? j1 : tiles);
      it->first = it->j0 == base;
      it->last = it->j1 == base + tiles;
      at += unit_len(p, tiles);
      if (prefix) {
        if (++rt == p.row_tiles_p) {
          rt = 0;
          if (++blk == p.blocks) {
            blk = 0;
            if (++h == H) { h = 0; prefix = false; }
          }
          measure(p, true);
        }
      } else if (n <= 0 || ++h == H) {
        h = 0;
        const bool other = n <= 0 || ++rt == p.row_tiles_s;
        if (other) { rt = 0; ++b; }
        measure(p, other);
      }
      if (it->j1 > it->j0) return true;
    }
    return false;
  }
};

// Row r of an item: its token (of B T), head within the group, keys seen; false past the rows.
__device__ __forceinline__ bool item_row(const Params& p, const Item& it, int r, int* token, int* g,
                                         int* lim) {
  const unsigned R = (unsigned)it.rt * kRows + r;     // rows are counted in 32 bits
  const int t = (int)(R / (unsigned)p.G);
  *g = (int)(R - (unsigned)t * p.G);
  if (it.prefix) {
    *token = t;
    *lim = p.a.prefix_len;
    return t < p.a.B * p.a.T;
  }
  *token = it.b * p.a.T + t;
  *lim = max(0, min(it.n, it.n - p.a.T + 1 + t));
  return t < p.a.T;
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (*abort) return false;
  if (mbar_wait_or_abort(bar, parity, abort)) return true;
  if (!*abort) atomicOr(&g_err_attn, kErrTimeout);
  *abort = 1;
  return false;
}

// What a score is multiplied with, in binary orders (a scale of zero goes into Q).
__host__ __device__ __forceinline__ float score_unit(float scale) {
  return scale == 0.0f ? 1.0f : fminf(fabsf(scale) * kLog2e, FLT_MAX);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t half2_to_e5m2(uint32_t a) {
  return __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&a), __NV_SATFINITE,
                                    __NV_E5M2);
}

// Four numbers of [0, 2^15] as sums of three e5m2 numbers (bytes of t0, t1, t2).  e5m2 is the
// upper byte of fp16, so a term is its fp16 number rounded at bit 8 (the differences are exact in
// fp16).  Rounding leaves a signed rest of at most half a unit, so three terms of three bits hold
// all eleven bits of fp16, down to e5m2's least number 2^-16.
__device__ __forceinline__ void split_e5m2(const float (&x)[4], uint32_t* t0, uint32_t* t1,
                                           uint32_t* t2) {
  constexpr uint32_t kHalf = 0x00800080u, kTop = 0xff00ff00u;
  const uint32_t a = pack_half(x[0], x[1]), b = pack_half(x[2], x[3]);
  const uint32_t ah = a + kHalf, bh = b + kHalf;
  const uint32_t ra = half2_sub(a, ah & kTop), rb = half2_sub(b, bh & kTop);
  const uint32_t am = ra + kHalf, bm = rb + kHalf;
  *t0 = __byte_perm(ah, bh, 0x7531);
  *t1 = __byte_perm(am, bm, 0x7531);
  *t2 = half2_to_e5m2(half2_sub(ra, am & kTop)) | half2_to_e5m2(half2_sub(rb, bm & kTop)) << 16;
}

__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  tmem_ld32(taddr, *reinterpret_cast<float(*)[32]>(&v[0]));
  tmem_ld32(taddr + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kThreads, 1)
    gdn_prefix_attention_kernel(const Params p, const __grid_constant__ CUtensorMap map_k,
                                const __grid_constant__ CUtensorMap map_v) {
  using Z = Shape<D, kF8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* sAbort = reinterpret_cast<volatile int*>(smem + Z::kMisc);
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + Z::kMisc + 4);
  int* sB0 = reinterpret_cast<int*>(smem + Z::kMisc + 8);
  long long* sAt0 = reinterpret_cast<long long*>(smem + Z::kMisc + 16);
  long long* sScan = reinterpret_cast<long long*>(smem + Z::kMax);   // 12 + 1 words, before use
  const uint32_t bar_full = sb + Z::kBars, bar_empty = bar_full + 8 * Z::kSlots;
  const uint32_t bar_s = bar_empty + 8 * Z::kSlots, bar_p = bar_s + 16, bar_pv = bar_p + 16;
  const uint32_t bar_q = bar_pv + 16, bar_xf = bar_q + 8, bar_xe = bar_xf + 16;
  const uint32_t bar_drain = bar_xe + 16;

  if (tid == 0) {
    for (int i = 0; i < Z::kSlots; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + 8 * i, 1);
      mbar_init(bar_p + 8 * i, kSoftmaxWarps);
      mbar_init(bar_pv + 8 * i, 1);
      mbar_init(bar_xf + 8 * i, 32);
      mbar_init(bar_xe + 8 * i, kSoftmaxWarps);
    }
    mbar_init(bar_q, kSoftmaxWarps);
    mbar_init(bar_drain, 1);
    fence_mbar_init();
    *sAbort = 0;
    *sB0 = p.a.B;
    *sAt0 = 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(sTmem), 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0 && p.a.cache.num_pages > 0) {   // (an empty cache has no maps)
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }

  // ---- the line: its length, then the sequence in which this CTA's part starts
  const long long w0 = tid < p.a.B ? seq_len_on_line(p, tid) : 0;   // the first kThreads of them
  long long sum = w0;
  for (int b = tid + kThreads; b < p.a.B; b += kThreads) sum += seq_len_on_line(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sScan[warp] = sum;
  __syncthreads();
  const long long wp = head_len(p) * p.a.cache.H;
  long long W = wp;
  for (int i = 0; i < kThreads / 32; ++i) W += sScan[i];
  const int parts = (int)(W < kCtas ? W : kCtas), c = blockIdx.x;
  const long long lo = parts > c ? W * c / parts : W, hi = parts > c ? W * (c + 1) / parts : W;
  const bool find = lo < hi && lo >= wp;
  if (find || c == 0) {
    long long carry = wp;
    for (int b0 = 0; b0 < p.a.B; b0 += kThreads) {
      const int b = b0 + tid;
      const long long w = b0 == 0 ? w0 : b < p.a.B ? seq_len_on_line(p, b) : 0;
      long long x = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();                                // sScan is read no more
      if (lane == 31) sScan[warp] = x;
      __syncthreads();
      long long before = carry;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += sScan[i];
        carry += sScan[i];
      }
      const long long at = before + x - w;
      if (find && at <= lo && lo < at + w) {
        *sB0 = b;
        *sAt0 = at;
      }
      if (c == 0 && b < p.a.B && p.a.kv_len[b] > (p.a.max_pages << p.a.cache.page_shift))
        atomicOr(&g_err_attn, kErrIndex);
      if (c != 0 && carry > lo) break;                // uniform
    }
  }
  pdl_trigger();                                      // the merge may be set up
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sTmem;
  Walk walk;
  walk.start(p, lo, hi, *sB0, *sAt0);
  Item it = {};

  if (warp == 0 || warp == 3) {
    // =================================================== producers: warp 0 K, warp 3 V.  The ring
    // holds, tile by tile of an item of n: K_0, K_1 V_0, K_2 V_1, ..., K_(n-1) V_(n-2), V_(n-1).
    const bool is_v = warp == 3;
    const CUtensorMap* map = is_v ? &map_v : &map_k;
    const int shift = p.a.cache.page_shift, per = kKeys >> shift, page = 1 << shift;
    const int head_rows = p.a.cache.H << shift;       // rows of a page, all heads
    const int outside = p.a.cache.num_pages * head_rows;
    uint32_t base = 0;                                // ring position of the item's first slot
    auto row_of = [&](int j) -> int {                 // of this lane's page of key tile j
      const int i = j * per + lane;
      if (lane >= per || (long long)i * page >= it.keys) return outside;
      if (!in_bounds(&g_err_attn, it.prefix ? (long long)i * page < p.a.prefix_len
                                            : it.b < p.a.B && i < p.a.max_pages))
        return outside;
      const int id = it.prefix ? p.a.prefix_pages[i]
                               : p.a.pages[(long long)it.b * p.a.max_pages + i];
      if ((unsigned)id >= (unsigned)p.a.cache.num_pages) {
        atomicOr(&g_err_attn, kErrIndex);
        return outside;
      }
      const int row = id * head_rows + (it.h << shift);
      return in_bounds(&g_err_attn, row >= 0 && row < outside) ? row : outside;
    };
    uint32_t last = 0;                                // ring position after this warp's last fill
    auto fill = [&](uint32_t ring, int row) {
#pragma unroll
      for (int s = 0; s < Z::kSlotsPerTile; ++s, ++ring) {
        const uint32_t slot = ring % Z::kSlots, use = ring / Z::kSlots;
        if (use > 0) wait(bar_empty + 8 * slot, (use - 1) & 1, sAbort);
        if (__any_sync(0xffffffffu, *sAbort)) return;
        if (lane == 0) mbar_arrive_expect_tx(bar_full + 8 * slot, Z::kSlotBytes);
        const uint32_t dst = sb + Z::kRing + slot * Z::kSlotBytes;
        __syncwarp();
        if (lane < per) {
#pragma unroll
          for (int k = 0; k < Z::kSlotBytes / (16 * KB); ++k)
            tma_load_3d(dst + k * 16 * KB + (lane << (shift + 7)), map,
                        (s * (Z::kSlotBytes / (16 * KB)) + k) * Z::kElem, row, 0,
                        bar_full + 8 * slot);
        }
        __syncwarp();
        last = ring + 1;
      }
    };
    while (walk.next(p, &it)) {
      const int n = it.j1 - it.j0;
      int row = row_of(it.j0);
      for (int i = 0; i < n; ++i) {
        const int after = i + 1 < n ? row_of(it.j0 + i + 1) : 0;
        const int pos = is_v ? min(2 * i + 2, 2 * n - 1) : max(2 * i - 1, 0);
        fill(base + pos * Z::kSlotsPerTile, row);
        row = after;
      }
      base += 2 * n * Z::kSlotsPerTile;
    }
    // after an abort: copies still in flight land before the CTA leaves (the other producer's
    // slots among these; a phase that never comes runs into the limit)
    if (__any_sync(0xffffffffu, *sAbort))
      for (uint32_t i = last > Z::kSlots ? last - Z::kSlots : 0; i < last; ++i)
        mbar_wait_bounded(bar_full + 8 * (i % Z::kSlots), (i / Z::kSlots) & 1, 1u << 12);
  } else if (warp == 1) {
    // =================================================== MMA issuer
    const bool leader = elect_one();
    const int page = 1 << p.a.cache.page_shift;
    uint32_t ring = 0, g = 0, items = 0;
    auto scores = [&](uint32_t gt) {
      const uint32_t d = tmem + TM_S + 128 * (gt & 1);
#pragma unroll
      for (int s = 0; s < Z::kSlotsPerTile; ++s, ++ring) {
        const uint32_t slot = ring % Z::kSlots, kb = sb + Z::kRing + slot * Z::kSlotBytes;
        if (!__all_sync(0xffffffffu, wait(bar_full + 8 * slot, (ring / Z::kSlots) & 1, sAbort)))
          return;
        tc_fence_after();
        if (leader) {
          if constexpr (kF8) {
            constexpr uint32_t id = idesc_f8(128, kKeys, 0, 0, false, false);
#pragma unroll
            for (int k = 0; k < 2 * (D / 32); ++k) {
              const int kk = k % (D / 32);
              mma_f8(d, sdesc_sw128(sb + (k / (D / 32)) * kRows * D + (kk >> 2) * 16 * KB + (kk & 3) * 32, 16, 1024),
                     sdesc_sw128(kb + (kk >> 2) * 16 * KB + (kk & 3) * 32, 16, 1024), id, k > 0);
            }
          } else {
            constexpr uint32_t id = idesc_bf16(128, kKeys, false, false);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_bf16(d, sdesc_sw128(sb + (2 * s + (k >> 2)) * 16 * KB + (k & 3) * 32, 16, 1024),
                       sdesc_sw128(kb + (k >> 2) * 16 * KB + (k & 3) * 32, 16, 1024), id,
                       s > 0 || k > 0);
          }
          mma_commit(bar_empty + 8 * slot);
          if (s == Z::kSlotsPerTile - 1) mma_commit(bar_s + 8 * (gt & 1));
        }
        __syncwarp();
      }
    };
    auto values = [&](uint32_t gt, int j, bool first) {
      const uint32_t a = tmem + TM_S + 128 * (gt & 1);
      if (!__all_sync(0xffffffffu, wait(bar_p + 8 * (gt & 1), (gt >> 1) & 1, sAbort))) return;
      const int live = it.keys - j * kKeys;           // rows of the tile that hold keys
#pragma unroll
      for (int s = 0; s < Z::kSlotsPerTile; ++s, ++ring) {
        const uint32_t slot = ring % Z::kSlots, vb = sb + Z::kRing + slot * Z::kSlotBytes;
        if (!__all_sync(0xffffffffu, wait(bar_full + 8 * slot, (ring / Z::kSlots) & 1, sAbort)))
          return;
        if (live < kKeys && (live & (page - 1))) {
          // the rest of the last page holds anything: zero it (0 * NaN)
          const int r1 = (live + page - 1) & ~(page - 1);
          for (int i = live * 8 + lane; i < r1 * 8; i += 32)
#pragma unroll
            for (int k = 0; k < Z::kSlotBytes / (16 * KB); ++k)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(vb + k * 16 * KB + i * 16),
                           "r"(0)
                           : "memory");
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (leader) {
          if constexpr (kF8) {
            constexpr uint32_t id = idesc_f8(128, D, 1, 0, false, true);
#pragma unroll
            for (int k = 0; k < 12; ++k)
              mma_f8_ta(tmem + TM_O, a + 32 * (k >> 2) + 8 * (k & 3),
                        sdesc_sw128(vb + (k & 3) * 4096, 16 * KB, 1024), id, !first || k > 0);
          } else {
            constexpr uint32_t id = idesc_bf16(128, 128, false, true);
#pragma unroll
            for (int k = 0; k < 16; ++k)                // P's two terms
              mma_bf16_ta(tmem + TM_O + 128 * s, a + 8 * k,
                          sdesc_sw128(vb + (k & 7) * 2048, 16 * KB, 1024), id, !first || k > 0);
          }
          mma_commit(bar_empty + 8 * slot);
          if (s == Z::kSlotsPerTile - 1) mma_commit(bar_pv + 8 * (gt & 1));
        }
        __syncwarp();
      }
    };
    while (walk.next(p, &it)) {
      wait(bar_q, items & 1, sAbort);
      ++items;
      scores(g);
      for (int j = it.j0 + 1; j < it.j1; ++j) {
        scores(g + 1);
        values(g, j - 1, j - 1 == it.j0);
        ++g;
      }
      values(g, it.j1 - 1, it.j1 - 1 == it.j0);
      ++g;
    }
    if (__any_sync(0xffffffffu, *sAbort)) {
      // after an abort: products in flight end before tensor memory is freed
      if (leader) mma_commit(bar_drain);
      __syncwarp();
      mbar_wait_bounded(bar_drain, 0);
    }
  } else if (warp == 2) {
    // =================================================== the 8-bit cache's scales
    if constexpr (kF8) {
      uint32_t g = 0;
      const int shift = p.a.cache.page_shift, pm = (1 << shift) - 1;
      while (walk.next(p, &it)) {
        for (int j = it.j0; j < it.j1; ++j, ++g) {
          const int key = j * kKeys + lane * 4;
          uint32_t ke = 0x7f7f7f7fu, ve = 0x7f7f7f7fu;  // 2^0 for keys that nothing sees
          if (key < it.keys) {
            const int i = key >> shift;
            const int id = it.prefix ? p.a.prefix_pages[i]
                                     : p.a.pages[(long long)it.b * p.a.max_pages + i];
            if ((unsigned)id < (unsigned)p.a.cache.num_pages) {
              const long long r = (((long long)id * p.a.cache.H + it.h) << shift) + (key & pm);
              if (in_bounds(&g_err_attn,
                            r + 4 <= ((long long)p.a.cache.num_pages * p.a.cache.H << shift))) {
                ke = *reinterpret_cast<const uint32_t*>(p.a.cache.k_exp + r);
                ve = *reinterpret_cast<const uint32_t*>(p.a.cache.v_exp + r);
              }
            }
          }
          float ks[4], ev[4], iv[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool live = key + e < it.keys;
            // exponents outside the format's range can only come from entries never written
            const int k = live ? min(max((int)(ke >> (8 * e) & 0xff), 67), 187) : 127;
            const int v = live ? min(max((int)(ve >> (8 * e) & 0xff), 67), 187) : 127;
            ks[e] = __uint_as_float((uint32_t)k << 23);
            ev[e] = (float)(v - 127);
            iv[e] = __uint_as_float((uint32_t)(254 - v) << 23);
          }
          const uint32_t st = g & 1;
          if (g >= 2) wait(bar_xe + 8 * st, ((g >> 1) - 1) & 1, sAbort);
          float4* dst = reinterpret_cast<float4*>(smem + Z::kScales + st * 1536) + lane;
          dst[0] = make_float4(ks[0], ks[1], ks[2], ks[3]);
          dst[32] = make_float4(ev[0], ev[1], ev[2], ev[3]);
          dst[64] = make_float4(iv[0], iv[1], iv[2], iv[3]);
          mbar_arrive(bar_xf + 8 * st);
        }
      }
    }
  } else if (warp >= 4) {
    // =================================================== softmax
    const int sw = warp - 4, quarter = sw & 3, half = sw >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    float* sMax = reinterpret_cast<float*>(smem + Z::kMax);
    float* sSum = reinterpret_cast<float*>(smem + Z::kSum);
    float* sQFac = reinterpret_cast<float*>(smem + Z::kQFac);
    // the scale's sign goes into Q, and so does a scale of zero
    const float coef = score_unit(p.a.scale);
    const uint32_t flip = p.a.scale < 0.0f ? 0x80008000u : 0u;
    // P may reach 2^kSlack over the reference: bf16 has fp32's range, so 32 leaves O and l far
    // from overflow and a raise to rows whose first tile says little; e5m2 ends at 57344, so the
    // reference lies kLift below the maximum and P starts at 2^kLift
    constexpr float kSlack = kF8 ? 7.0f : 32.0f, kLift = kF8 ? 8.0f : 0.0f;
    // turn: counts the items (a warp may load the next one's Q while another has yet to read its
    // own row's factor of this one)
    uint32_t g = 0, turn = 0;
    // Q: an item's rows, dealt to the warps and gathered into the swizzled K-major layout (small
    // loops: this code runs once an item and its instructions come from L2).  8-bit: a row's
    // bf16 elements land where its two terms will lie, 4 x 128 bytes, and are split in place.
    auto load_q = [&](const Item& it) {
      constexpr int L = D / 8, kPer = 32 / L;         // lanes a row, rows a pass
      const int ql = lane % L;
      const long long left = (long long)(it.prefix ? p.a.B : 1) * p.a.T * p.G -
                             (long long)it.rt * kRows;
      const int n = left < kRows ? (int)left : kRows;   // (rows past them feed no live row)
      auto at = [&](int row) {                        // this lane's 16 bytes of a bf16 row
        return (uint32_t)((ql >> 3) * 16 * KB + row * 128 + (((ql & 7) ^ (row & 7)) << 4));
      };
      {
        int row = sw * kPer + lane / L;
        const unsigned R = (unsigned)it.rt * kRows + row;
        unsigned t = R / (unsigned)p.G, gh = R - t * p.G;
        const unsigned dt = 8 * kPer / (unsigned)p.G, dg = 8 * kPer - dt * p.G;   // a pass further
        const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(p.a.q) +
                                  (it.prefix ? 0ll : (long long)it.b * p.a.T) * p.a.q_stride +
                                  (long long)it.h * p.G * D + ql * 8;
#pragma unroll 2
        for (; row < n; row += 8 * kPer) {
          if (in_bounds(&g_err_attn, (it.prefix ? 0 : it.b) * p.a.T + (int)t < p.a.B * p.a.T &&
                                         it.h * p.G + (int)gh < p.a.Hq && row < kRows))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(sb + at(row)),
                         "l"(q0 + t * p.a.q_stride + gh * D)
                         : "memory");
          gh += dg;
          t += dt;
          if (gh >= (unsigned)p.G) gh -= p.G, ++t;
        }
      }
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      if (p.a.scale == 0.0f) {
        // zero times Q: NaN is left where an element is not finite
        auto times0 = [](uint32_t w) -> uint32_t {
          return ((w & 0x7f80u) == 0x7f80u ? 0x7fc0u : 0u) |
                 ((w & 0x7f800000u) == 0x7f800000u ? 0x7fc00000u : 0u);
        };
#pragma unroll 1
        for (int row = sw * kPer + lane / L; row < n; row += 8 * kPer) {
          uint4* u = reinterpret_cast<uint4*>(smem + at(row));
          *u = make_uint4(times0(u->x), times0(u->y), times0(u->z), times0(u->w));
        }
      }
      if (kF8 || p.a.scale < 0.0f) {
        constexpr int kAt = 4;                        // passes side by side
#pragma unroll 1
        for (int r0 = sw * kPer; r0 < n; r0 += kAt * 8 * kPer) {
          uint32_t w[kAt][4];
          float top[kAt];
#pragma unroll
          for (int i = 0; i < kAt; ++i) {
            const int row = r0 + i * 8 * kPer + lane / L;
            const uint4 u = row < n ? *reinterpret_cast<const uint4*>(smem + at(row))
                                    : make_uint4(0, 0, 0, 0);
            w[i][0] = u.x ^ flip; w[i][1] = u.y ^ flip;
            w[i][2] = u.z ^ flip; w[i][3] = u.w ^ flip;
            if (!kF8 && row < n)
              *reinterpret_cast<uint4*>(smem + at(row)) =
                  make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            top[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top[i] = fmaxf(top[i], fmaxf(fabsf(__uint_as_float(w[i][e] << 16)),
                                           fabsf(__uint_as_float(w[i][e] & 0xffff0000u))));
          }
          if constexpr (kF8) {
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
              for (int i = 0; i < kAt; ++i)
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
            __syncwarp();                             // the passes' rows are read
#pragma unroll
            for (int i = 0; i < kAt; ++i) {
              const int row = r0 + i * 8 * kPer + lane / L;
              // 2^-e with top 2^-e of [224, 448]; e kept where both powers are normal
              const uint32_t bits = __float_as_uint(top[i]);
              int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
              e = min(max(e, -120), 120);
              // (an infinite query makes its row NaN)
              const float f = top[i] < INFINITY ? __uint_as_float((uint32_t)(127 - e) << 23) : NAN;
              uint32_t hw[4], lw[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float a0 = __uint_as_float(w[i][q] << 16) * f;
                const float a1 = __uint_as_float(w[i][q] & 0xffff0000u) * f;
                // the leading four bits by Veltkamp's splitting, 24 - 20 of fp32's
                const float c0 = a0 * 1048577.0f, c1 = a1 * 1048577.0f;
                const float h0 = __fsub_rn(c0, __fsub_rn(c0, a0)), h1 = __fsub_rn(c1, __fsub_rn(c1, a1));
                hw[q] = __nv_cvt_float2_to_fp8x2(make_float2(h0, h1), __NV_SATFINITE, __NV_E4M3);
                lw[q] = __nv_cvt_float2_to_fp8x2(make_float2(a0 - h0, a1 - h1), __NV_SATFINITE,
                                                 __NV_E4M3);
              }
              if (row < n) {
                uint8_t* to = smem + (ql >> 4) * 16 * KB + row * 128 +
                              ((((ql & 15) >> 1) ^ (row & 7)) << 4) + (ql & 1) * 8;
                *reinterpret_cast<uint2*>(to) = make_uint2(hw[0] | hw[1] << 16, hw[2] | hw[3] << 16);
                *reinterpret_cast<uint2*>(to + kRows * D) =
                    make_uint2(lw[0] | lw[1] << 16, lw[2] | lw[3] << 16);
                if (ql == 0)
                  sQFac[128 * (turn & 1) + row] = __uint_as_float((uint32_t)(127 + e) << 23);
              }
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q);
      if constexpr (kF8) named_bar_sync(5, 32 * kSoftmaxWarps);
    };
    // Each turn takes the next item's Q first (every score of the item before is done), so that
    // its first scores run beside the end of the item before; its first P waits for this
    // thread, so O stays until then.
    bool live = false, any_live = false;
    float m = -INFINITY, l = 0.0f;                    // reference, this half's sum
    // bf16: the score whose product with rc m is, and whether m is large in a row of the warp: an
    // m past kNear rounds by more than 2^x takes, and the reference is the product itself
    float from = -INFINITY;
    bool any_far = false;
    for (bool begun = false;; begun = true, ++turn) {
      const Item done = it;
      const bool more = walk.next(p, &it);
      if (more) load_q(it);
      // ---- the part: O, m, l of the item's rows
      if (begun) wait(bar_pv + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, sAbort);
      if (begun && r == 0 && half == 0 && in_workspace(p, done.prefix, done.unit, c, 0)) {
        // where the merge finds the unit's parts
        int2* span = (done.prefix ? p.span_p : p.span_s) + done.unit;
        if (done.first) span->x = c;
        if (done.last) span->y = c;
      }
      if (begun && any_live) {
        tc_fence_after();
        if (half == 1) sSum[r] = l;
        named_bar_sync(1 + quarter, 64);
        if (half == 0) l += sSum[r];
        // lanes hold consecutive rows: 16 bytes a row side by side
        const int stored = done.prefix ? p.rows_p : p.rows_s;
        const long long slot = done.unit + c;
        float4* op = reinterpret_cast<float4*>(done.prefix ? p.o_p : p.o_s) +
                     (slot * (D / 4) + half * (D / 8)) * stored + r;
#pragma unroll 1
        for (int i = 0; i < D / 8; i += 8) {
          float o[32];
          tmem_ld32(tmem + TM_O + lane_base + half * (D / 2) + 4 * i, o);
          tmem_wait_ld();
          if (live && in_workspace(p, done.prefix, done.unit, c, r)) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              op[(long long)(i + e) * stored] =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        // m = -inf says that the row saw nothing; a row of NaN scores did
        if (live && half == 0 && in_workspace(p, done.prefix, done.unit, c, r)) {
          // (a score beyond what fp32 holds is still one)
          const float ref = kF8 || from == -INFINITY ? m : fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
          (done.prefix ? p.ml_p : p.ml_s)[slot * stored + r] = make_float2(l == l ? ref : 0.0f, l);
          if (!kF8 && fabsf(ref) > kFar) (done.prefix ? p.far_p : p.far_s)[slot * stored + r] = from;
        }
        tc_fence_before();
      }
      if (!more) break;
      // ---- the item's tiles
      int token, gh, lim;
      live = item_row(p, it, r, &token, &gh, &lim);
      if (!live) lim = 0;
      any_live = __any_sync(0xffffffffu, live);
      const float rc = kF8 ? coef * sQFac[128 * (turn & 1) + r] : coef;
      const unsigned long long rc2 = pair(rc, rc);
      m = -INFINITY;
      l = 0.0f;
      for (int j = it.j0; j < it.j1; ++j, ++g) {
        const uint32_t buf = g & 1, ts = tmem + TM_S + 128 * buf + lane_base;
        wait(bar_s + 8 * buf, (g >> 1) & 1, sAbort);
        if constexpr (kF8) wait(bar_xf + 8 * buf, (g >> 1) & 1, sAbort);
        if (any_live) {
          tc_fence_after();
          float s[64];
          tmem_ld64(ts + 64 * half, s);
          tmem_wait_ld();
          const float4* ks = reinterpret_cast<const float4*>(smem + Z::kScales + buf * 1536) + 16 * half;
          if constexpr (kF8) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 k4 = ks[i], v4 = ks[32 + i];
              unpair(fma2(mul2(pair(s[4 * i], s[4 * i + 1]), pair(k4.x, k4.y)), rc2,
                          pair(v4.x, v4.y)), &s[4 * i], &s[4 * i + 1]);
              unpair(fma2(mul2(pair(s[4 * i + 2], s[4 * i + 3]), pair(k4.z, k4.w)), rc2,
                          pair(v4.z, v4.w)), &s[4 * i + 2], &s[4 * i + 3]);
            }
          }
          const int seen = lim - j * kKeys - 64 * half;  // this half's keys that the row sees
          if (__any_sync(0xffffffffu, seen < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= seen) s[i] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 64; i += 4) {
            mx[0] = fmaxf(mx[0], s[i]);
            mx[1] = fmaxf(mx[1], s[i + 1]);
            mx[2] = fmaxf(mx[2], s[i + 2]);
            mx[3] = fmaxf(mx[3], s[i + 3]);
          }
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          float* sm = sMax + buf * 256;
          sm[half * 128 + r] = top;
          named_bar_sync(1 + quarter, 64);
          top = fmaxf(top, sm[(1 - half) * 128 + r]);
          const float score = top;
          if constexpr (!kF8) top *= rc;
          // the reference: the first maximum; later only when it is passed by more than kSlack
          bool raise = kF8 ? top - m > kLift + kSlack : top > m + kSlack;
          if (!kF8 && any_far && fabsf(m) > kNear)
            raise = scaled_difference(score, from, rc) > kSlack;
          auto lifted = [&]() {                       // (a large maximum less kLift would round)
            return !kF8 ? top : fabsf(top) > kNear ? top : top - kLift;
          };
          if (j == it.j0) {
            m = lifted();
            if constexpr (!kF8) {
              from = score;
              any_far = __any_sync(0xffffffffu, fabsf(m) > kNear && score != -INFINITY);
            }
          } else if (__any_sync(0xffffffffu, raise)) {
            const float mn = raise ? lifted() : m;
            float f = raise ? ex2_approx(m - mn) : 1.0f;
            m = mn;
            if constexpr (!kF8) {
              if (raise) {
                if (any_far || fabsf(m) > kNear) f = ex2_approx(reference_difference(from, score, rc));
                from = score;
              }
              any_far = __any_sync(0xffffffffu, fabsf(m) > kNear && from != -INFINITY);
            }
            l *= f;
            wait(bar_pv + 8 * (buf ^ 1), ((g - 1) >> 1) & 1, sAbort);  // O of the tiles before
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D / 2; i += 32) {
              float o[32];
              const uint32_t to = tmem + TM_O + lane_base + half * (D / 2) + i;
              tmem_ld32(to, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st32(to, o);
            }
            tmem_wait_st();
          }
          float base = (kF8 ? m : from) == -INFINITY ? 0.0f : m;
          if constexpr (!kF8) {
            // s rc - m in one rounding; in the rows of a large m (s - from) rc
            if (any_far) {
              const bool far = fabsf(base) > kNear;
              const float sub = far ? -from : 0.0f;
              const unsigned long long minus_from = pair(sub, sub);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                unpair(add2(pair(s[2 * i], s[2 * i + 1]), minus_from), &s[2 * i], &s[2 * i + 1]);
              if (far) base = 0.0f;
            }
          }
          const unsigned long long minus_base = pair(-base, -base);
          unsigned long long sum2[2] = {};            // pairs
          if constexpr (kF8) {
            uint32_t t0[16], t1[16], t2[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 iv = ks[64 + i];
              float e[4];
              unpair(add2(pair(s[4 * i], s[4 * i + 1]), minus_base), &e[0], &e[1]);
              unpair(add2(pair(s[4 * i + 2], s[4 * i + 3]), minus_base), &e[2], &e[3]);
#pragma unroll
              for (int q = 0; q < 4; ++q) e[q] = ex2_approx(e[q]);
              sum2[0] = fma2(pair(e[0], e[1]), pair(iv.x, iv.y), sum2[0]);
              sum2[1] = fma2(pair(e[2], e[3]), pair(iv.z, iv.w), sum2[1]);
              split_e5m2(e, &t0[i], &t1[i], &t2[i]);
            }
            tmem_st16(ts + 16 * half, t0);
            tmem_st16(ts + 32 + 16 * half, t1);
            tmem_st16(ts + 64 + 16 * half, t2);
          } else {
            float hi[32], lo[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float e0, e1;
              unpair(fma2(pair(s[2 * i], s[2 * i + 1]), rc2, minus_base), &e0, &e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              const unsigned long long e2 = pair(e0, e1);
              sum2[i & 1] = add2(sum2[i & 1], e2);
              // the leading bits by truncation, the exact rest rounded
              const float h0 = __uint_as_float(__float_as_uint(e0) & 0xffff0000u);
              const float h1 = __uint_as_float(__float_as_uint(e1) & 0xffff0000u);
              hi[i] = __uint_as_float(__byte_perm(__float_as_uint(e0), __float_as_uint(e1), 0x7632));
              float l0, l1;
              unpair(add2(e2, pair(-h0, -h1)), &l0, &l1);
              lo[i] = __uint_as_float(pack_bf16(l0, l1));
            }
            tmem_st32(ts + 32 * half, hi);
            tmem_st32(ts + 64 + 32 * half, lo);
          }
          float l4[4];
          unpair(sum2[0], &l4[0], &l4[1]);
          unpair(sum2[1], &l4[2], &l4[3]);
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_p + 8 * buf);
          if constexpr (kF8) mbar_arrive(bar_xe + 8 * buf);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------------- the merge

// A row whose references are so large that their rounding shows: its parts joined by the scores
// that these are of, one after the other.  One 16-byte vector (cg) of row R of head h.
template <int D>
__device__ __noinline__ void join_far(const Params& p, int b, int h, unsigned R, int rs, bool own,
                                      int cg, float4* acc, float* m, float* l) {
  const int rt_p = (int)(R / kRows), rt_s = rs / kRows;
  float top = -INFINITY;
  for (int pass = 0; pass < 2; ++pass) {
    auto unit = [&](bool prefix, int2 span, long long u, const float* o, const float2* ml,
                    const float* far, int stored, int r) {
      span.y = min(span.y, kCtas - 1);
      for (int c = max(span.x, 0); c <= span.y; ++c) {
        if (!in_workspace(p, prefix, u, c, r)) break;
        const long long at = (u + c) * stored + r;
        const float2 v = ml[at];
        if (v.x == -INFINITY) continue;
        const bool counts = fabsf(v.x) > kFar;        // the others weigh nothing (NaN stays)
        if (pass == 0) {
          if (counts) top = fmaxf(top, far[at]);
          continue;
        }
        const float w = counts ? ex2_approx(reference_difference(far[at], top, p.coef)) : 0.0f;
        const float4 x =
            reinterpret_cast<const float4*>(o)[((u + c) * (D / 4) + cg) * stored + r];
        *l += v.y * w;
        acc->x += x.x * w; acc->y += x.y * w; acc->z += x.z * w; acc->w += x.w * w;
      }
    };
    if (pass == 1) {
      *acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      *l = 0.0f;
    }
    for (int blk = 0; p.prefix_tiles > 0 && blk < p.blocks; ++blk) {
      const long long u = ((long long)h * p.blocks + blk) * p.row_tiles_p + rt_p;
      unit(true, p.span_p[u], u, p.o_p, p.ml_p, p.far_p, p.rows_p, R % kRows);
    }
    const long long u = ((long long)b * p.row_tiles_s + rt_s) * p.a.cache.H + h;
    if (own) unit(false, p.span_s[u], u, p.o_s, p.ml_s, p.far_s, p.rows_s, rs % kRows);
  }
  *m = top * p.coef;
}

// A warp takes eight rows of one head (the parts lie with consecutive rows side by side) and 64
// columns, and joins the rows' parts: the CTAs of a unit's span, one slot each.  Few rows are cut
// into many parts: then (kGroups = 8) the eight warps of a block share out the parts of the same
// rows, so that they are read at the same time, and join what they have in shared memory.  Bound
// by the latency of the parts' loads, out of L2: 5 to 8 us of the whole.
//
// The bounds keep the bf16 cache's code at 80 registers, three blocks an SM (128 sequences, D = 128:
// 48.3 us; with 64 registers 51.0).
template <int D, typename Tout, int kGroups, int kAhead, bool kF8>
__global__ void __launch_bounds__(256, kF8 ? 0 : kAhead == 4 ? 2 : 3)
    gdn_prefix_merge_kernel(const Params p) {
  constexpr int kVec = 4;                             // 16-byte vectors a lane
  __shared__ float4 s_acc[kGroups][16][8];            // [warp][vector of the 64 columns][row]
  __shared__ float2 s_ml[kGroups][8];
  const unsigned rows = (unsigned)p.a.B * p.a.T * p.G;   // of a head
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane & 7;
  const int group = kGroups == 1 ? 0 : warp;
  const unsigned R0 = (kGroups == 1 ? blockIdx.x * 8u + warp : blockIdx.x) * 8u + r8, R = R0 < rows ? R0 : rows - 1;
  const int cg = blockIdx.z * 16 + (lane >> 3), h = blockIdx.y, H = p.a.cache.H;
  const int token = (int)(R / (unsigned)p.G), gh = (int)(R - (unsigned)token * p.G);
  const int b = token / p.a.T, t = token - b * p.a.T;
  const int raw = p.a.kv_len[b], n = own_len(p.a, b);
  const int rs = t * p.G + gh, rt_s = rs / kRows, rt_p = (int)(R / kRows);
  const bool own = n > 0 && tile_keys(p, n, rt_s) > 0;
  const long long unit_s = ((long long)b * p.row_tiles_s + rt_s) * H + h;
  pdl_wait();
  float acc[4 * kVec] = {}, m = -INFINITY, l = 0.0f;
  // the parts span.x + skip, + step, ... of a unit
  auto join = [&](bool prefix, int2 span, long long unit, const float* o, const float2* ml,
                  int stored, int r, int skip, int step) {
    span.y = min(span.y, kCtas - 1);                  // (whatever a spoilt workspace says)
    if (!in_workspace(p, prefix, unit, 0, r)) return;
    for (int c = max(span.x, 0) + skip; c <= span.y; c += kAhead * step) {
      float2 v[kAhead];
      float4 x[kAhead][kVec];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const long long slot = unit + min(c + i * step, span.y);
        const float4* src = reinterpret_cast<const float4*>(o) + (slot * (D / 4) + cg) * stored + r;
        v[i] = ml[slot * stored + r];
#pragma unroll
        for (int q = 0; q < kVec; ++q) x[i][q] = src[(long long)(4 * q) * stored];
        if (c + i * step > span.y) v[i] = make_float2(-INFINITY, 0.0f);
      }
      float mn = m;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) mn = fmaxf(mn, v[i].x);
      if (mn == -INFINITY) continue;                  // no key seen
      const float f = ex2_approx(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int e = 0; e < 4 * kVec; ++e) acc[e] *= f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (v[i].x == -INFINITY) continue;            // its O holds nothing
        const float w = ex2_approx(v[i].x - mn);
        l += v[i].y * w;
#pragma unroll
        for (int q = 0; q < kVec; ++q) {
          acc[4 * q] += x[i][q].x * w;
          acc[4 * q + 1] += x[i][q].y * w;
          acc[4 * q + 2] += x[i][q].z * w;
          acc[4 * q + 3] += x[i][q].w * w;
        }
      }
    }
  };
  if (raw >= 0) {
    const int2 span_s =
        own && in_workspace(p, false, unit_s, 0, 0) ? p.span_s[unit_s] : make_int2(0, -1);
    if (p.prefix_tiles > 0) {
      // a warp takes whole blocks, or parts of each
      const bool whole = p.blocks >= kGroups;
      for (int blk = whole ? group : 0; blk < p.blocks; blk += whole ? kGroups : 1) {
        const long long unit = ((long long)h * p.blocks + blk) * p.row_tiles_p + rt_p;
        if (!in_workspace(p, true, unit, 0, 0)) break;
        join(true, p.span_p[unit], unit, p.o_p, p.ml_p, p.rows_p, R % kRows,
             whole ? 0 : (group + blk) % kGroups, whole ? 1 : kGroups);
      }
    }
    join(false, span_s, unit_s, p.o_s, p.ml_s, p.rows_s, rs % kRows, (group + kGroups / 2) % kGroups,
         kGroups);
  }
  const long long row = (long long)token * p.a.Hq + h * p.G + gh;
  Tout* out = static_cast<Tout*>(p.a.out) + row * D + blockIdx.z * 64;
  const bool lead = blockIdx.z == 0;
  // (twice kFar: what lies below kFar then weighs nothing)
  auto far = [&]() { return !kF8 && fabsf(m) > 2.0f * kFar && m != -INFINITY; };
  auto store = [&](int vec, const float* y) {
    if (!in_bounds(&g_err_attn, row < (long long)p.a.B * p.a.T * p.a.Hq &&
                                    (int)blockIdx.z * 64 + 4 * vec + 4 <= D))
      return;
    // l is NaN where a score is, 0 where no key is seen
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if constexpr (sizeof(Tout) == 2)
      *reinterpret_cast<uint2*>(out + 4 * vec) =
          make_uint2(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv));
    else
      *reinterpret_cast<float4*>(out + 4 * vec) =
          make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    if (p.a.lse && lead && vec == 0)
      p.a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  };
  if constexpr (kGroups == 1) {
    if (R0 >= rows) return;
    if (far()) {
      float4 x;
      float m1, l1;
#pragma unroll 1
      for (int q = 0; q < kVec; ++q) {
        join_far<D>(p, b, h, R, rs, own, cg + 4 * q, &x, &m1, &l1);
        m = m1, l = l1;
        const float y[4] = {x.x, x.y, x.z, x.w};
        store(4 * q + (lane >> 3), y);
      }
      return;
    }
#pragma unroll
    for (int q = 0; q < kVec; ++q) store(4 * q + (lane >> 3), acc + 4 * q);
  } else {
#pragma unroll
    for (int q = 0; q < kVec; ++q)
      s_acc[warp][4 * q + (lane >> 3)][r8] =
          make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
    if (lane < 8) s_ml[warp][lane] = make_float2(m, l);
    __syncthreads();
    // 128 threads: a row and a 16-byte vector of the 64 columns each
    const int vec = threadIdx.x >> 3;
    if (threadIdx.x >= 128 || R0 >= rows) return;
    float2 v[kGroups];
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      v[i] = s_ml[i][r8];
      m = fmaxf(m, v[i].x);
    }
    l = 0.0f;
    float y[4] = {};
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      if (v[i].x == -INFINITY) continue;
      const float w = ex2_approx(v[i].x - m);
      const float4 x = s_acc[i][vec][r8];
      l += v[i].y * w;
      y[0] += x.x * w; y[1] += x.y * w; y[2] += x.z * w; y[3] += x.w * w;
    }
    if (far()) {
      float4 x;
      float m1, l1;
      join_far<D>(p, b, h, R, rs, own, blockIdx.z * 16 + vec, &x, &m1, &l1);
      m = m1, l = l1;
      y[0] = x.x, y[1] = x.y, y[2] = x.z, y[3] = x.w;
    }
    store(vec, y);
  }
}

template <int D, typename Tout, bool kF8>
cudaError_t launch_merge(const Params& p, cudaStream_t stream) {
  const long long eights = ((long long)p.a.B * p.a.T * p.G + 7) / 8;
  const unsigned H = (unsigned)p.a.cache.H, Z = D / 64;
  // kAhead parts in flight a warp: four where all blocks are resident at 128 registers a thread
  // (32 sequences, 16384 shared tokens, 384 blocks: 43.2 us with four, 41.5 with two; 16
  // sequences, 192 blocks: 29.3 and 30.5)
  if (eights * H * Z <= 2 * kCtas)
    return launch_pdl(true, gdn_prefix_merge_kernel<D, Tout, 8, 4, kF8>, dim3((unsigned)eights, H, Z),
                      dim3(256), 0, stream, p);
  if (eights * H <= kFewRows / 8)
    return launch_pdl(true, gdn_prefix_merge_kernel<D, Tout, 8, 2, kF8>, dim3((unsigned)eights, H, Z),
                      dim3(256), 0, stream, p);
  return launch_pdl(true, gdn_prefix_merge_kernel<D, Tout, 1, 2, kF8>,
                    dim3((unsigned)((eights + 7) / 8), H, Z), dim3(256), 0, stream, p);
}

// ------------------------------------------------------------------------------- host side

struct Layout {
  int row_tiles_p, row_tiles_s, rows_p, rows_s;
  size_t span_p, span_s, ml_p, ml_s, far_p, far_s, o_p, o_s, total;
};

Layout layout_of(int B, int T, int Hq, int H, int D) {
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  Layout y;
  const int G = Hq / H;
  const long long rp = (long long)B * T * G, rs = (long long)T * G;
  y.row_tiles_p = (int)((rp + kRows - 1) / kRows);
  y.row_tiles_s = (int)((rs + kRows - 1) / kRows);
  y.rows_p = (int)(rp < kRows ? rp : kRows);
  y.rows_s = (int)(rs < kRows ? rs : kRows);
  size_t up_units = (size_t)H * y.row_tiles_p;        // at most kCtas more of them by blocks
  if (up_units < kCtas) up_units = kCtas;
  const size_t np = (up_units + kCtas) * y.rows_p;
  const size_t ns = ((size_t)B * y.row_tiles_s * H + kCtas) * y.rows_s;
  size_t off = 0;
  y.span_p = off; off += up(8 * up_units);
  y.span_s = off; off += up(8 * (size_t)B * y.row_tiles_s * H);
  y.ml_p = off; off += up(8 * np);
  y.ml_s = off; off += up(8 * ns);
  y.far_p = off; off += up(4 * np);
  y.far_s = off; off += up(4 * ns);
  y.o_p = off; off += up(4 * np * D);
  y.o_s = off; off += up(4 * ns * D);
  y.total = off;
  return y;
}

template <int D, bool kF8>
cudaError_t launch(const Params& p, cudaStream_t stream) {
  using Z = Shape<D, kF8>;
  const GdnKvCacheArgs& c = p.a.cache;
  static unsigned done = 0;
  cudaError_t e = set_smem_once(gdn_prefix_attention_kernel<D, kF8>, Z::kBytes, &done);
  if (e != cudaSuccess) return e;
  CUtensorMap mk = {}, mv = {};
  if (c.num_pages > 0) {
    const CUtensorMapDataType dt =
        kF8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int rows = c.num_pages * (c.H << c.page_shift);
    if (!gdn_make_map(&mk, c.k, dt, kF8 ? 1 : 2, D, rows, 1, D, Z::kElem, 1 << c.page_shift, true) ||
        !gdn_make_map(&mv, c.v, dt, kF8 ? 1 : 2, D, rows, 1, D, Z::kElem, 1 << c.page_shift, true))
      return cudaErrorInvalidValue;
  }
  e = launch_pdl(false, gdn_prefix_attention_kernel<D, kF8>, dim3(kCtas), dim3(kThreads), Z::kBytes,
                 stream, p, mk, mv);
  if (e != cudaSuccess) return e;
  return p.a.out_bf16 ? launch_merge<D, __nv_bfloat16, kF8>(p, stream)
                       : launch_merge<D, float, kF8>(p, stream);
}

}  // namespace

size_t gdn_prefix_attention_bytes(int B, int T, int Hq, int H, int D) {
  return layout_of(B, T, Hq, H, D).total;
}

cudaError_t gdn_launch_prefix_attention(const GdnAttnArgs& a, cudaStream_t stream) {
  const Layout y = layout_of(a.B, a.T, a.Hq, a.cache.H, a.cache.D);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  Params p;
  p.a = a;
  p.G = a.Hq / a.cache.H;
  p.row_tiles_p = y.row_tiles_p;
  p.row_tiles_s = y.row_tiles_s;
  p.prefix_tiles = (a.prefix_len + kKeys - 1) / kKeys;
  // Several row tiles of a prefix far larger than L2: blocks of keys of about one CTA's part, so
  // that the row tiles read the same keys at the same time.  Smaller ones stay in L2 long enough,
  // and blocks cost more parts to join (16 x 4 tokens, bf16, 134 MB of prefix: 75 us with, 71
  // without; 40 x 4: 183, 157; 12 x 4 tokens, 537 MB: 223, 250; 40 x 4, 410 MB: 459, 478).
  const long long prefix_bytes = 2ll * a.prefix_len * a.cache.H * a.cache.D * (a.cache.f8 ? 1 : 2);
  p.blocks = 1;
  if (y.row_tiles_p > 1 && prefix_bytes > kBlockBytes) {
    p.blocks = kCtas / (y.row_tiles_p * a.cache.H);
    if (p.blocks < 1) p.blocks = 1;
    if (p.blocks > p.prefix_tiles) p.blocks = p.prefix_tiles;
  }
  p.block_tiles = p.prefix_tiles ? (p.prefix_tiles + p.blocks - 1) / p.blocks : 1;
  if (p.prefix_tiles) p.blocks = (p.prefix_tiles + p.block_tiles - 1) / p.block_tiles;
  // about 2.5 us: a tile of 128 KB, two of less (measured at 1 / 2: 128 sequences with tails of
  // 1000 tokens, bf16, D = 256: 110 / 117 us; the same at D = 128: 70 / 67; prompt of 666 tokens
  // on 20000, D = 128: 162 / 143; 32 sequences on 16384, 8-bit, D = 256: 44 / 43)
  p.unit_cost = a.cache.D == 256 && !a.cache.f8 ? 1 : 2;
  p.coef = score_unit(a.scale);
  p.rows_p = y.rows_p;
  p.rows_s = y.rows_s;
  p.span_p = reinterpret_cast<int2*>(ws + y.span_p);
  p.span_s = reinterpret_cast<int2*>(ws + y.span_s);
  p.ml_p = reinterpret_cast<float2*>(ws + y.ml_p);
  p.ml_s = reinterpret_cast<float2*>(ws + y.ml_s);
  p.far_p = a.cache.f8 ? nullptr : reinterpret_cast<float*>(ws + y.far_p);
  p.far_s = a.cache.f8 ? nullptr : reinterpret_cast<float*>(ws + y.far_s);
  p.o_p = reinterpret_cast<float*>(ws + y.o_p);
  p.o_s = reinterpret_cast<float*>(ws + y.o_s);
  if (a.cache.D == 128)
    return a.cache.f8 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return a.cache.f8 ? launch<256, true>(p, stream) : launch<256, false>(p, stream);
}
