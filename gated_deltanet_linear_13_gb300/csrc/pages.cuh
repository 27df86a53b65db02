// Pages, slots and positions of a step's new tokens, and pages given back, from the requests'
// lengths on the device.
//
// Both calls are a scan over the B requests (tokens and pages that each adds or gives back), a few
// words a token or table entry behind it, and the new state of the pool.  The scan is a microsecond,
// so every CTA does it for itself and takes its share of the rest.  The pool's counts must not change
// before the last CTA has read them: the CTAs of one cluster meet at its barrier, which is one
// launch; a large step writes its outputs with many CTAs and the state in a second launch, set up
// beside the first.  Nothing is kept between calls.  Bound by latency: a launch (2.2 us), two loads
// that depend on each other, the barrier and a table entry's load: 3.5 us a call for 64 requests.
// Part of kv_cache.cu, whose error word it uses.
#pragma once

#include <algorithm>

#include "common.cuh"

using namespace gdn;

namespace {
namespace pages {

constexpr int kMostThreads = 1024, kMostWarps = kMostThreads / 32;
constexpr int kMaxCtas = 8;                // of the cluster (the portable most)
constexpr int kAtOnce = 4;                 // entries of a block table on the way in a lane
// Words of output up to which one cluster does everything; above, many CTAs write the outputs and a
// second launch the state (a plan and a release: 20000 tokens 10.3 us in one cluster, 9.2 in two
// launches; 80000 13.1 / 9.5; 240000 21.9 / 10.7).
constexpr long long kOneCluster = 16384;
constexpr int kInRow = 4;                  // tokens of a lane, 32 apart

struct Shared {                            // [B + 1] and [B]
  int* tokens;                             // first packed token of each request, then their number
  int* pages;                              // first page (of those taken or given) of each
  int* row;                                // -1: left out
  int* held;
  int* from;                               // plan: kv_len; release: pages kept
};

__device__ __forceinline__ Shared carve(int* smem, int B) {
  return Shared{smem, smem + B + 1, smem + 2 * B + 2, smem + 3 * B + 2, smem + 4 * B + 2};
}
size_t shared_bytes(int B) { return sizeof(int) * (5 * (size_t)B + 2); }

struct WarpSums {                          // of a scan: the running sums, and the totals in halves
  unsigned a, b, a_low, a_high, b_low, b_high;
};
// Dynamic shared memory that a kernel may have without asking for more: 48 KB with what it declares.
constexpr size_t kUnasked = 48 * 1024 - kMostWarps * sizeof(WarpSums);

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int r;
  asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Two numbers below 2^31 a thread: their sums over the threads before this one (modulo 2^32, right
// where the totals are below that), and the block's exact totals.
struct Two {
  unsigned a, b;
};
struct Totals {
  unsigned long long a, b;
};
__device__ __forceinline__ Two scan(Two x, Totals* totals) {
  __shared__ WarpSums s_warp[kMostWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  constexpr unsigned kAll = 0xffffffffu;
  auto inclusive = [&](Two v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned a = __shfl_up_sync(kAll, v.a, o), b = __shfl_up_sync(kAll, v.b, o);
      if (lane >= o) v.a += a, v.b += b;
    }
    return v;
  };
  const Two sum = inclusive(x);
  // (in halves, whose sums over 8192 requests stay below 2^32)
  const WarpSums mine{0, 0, __reduce_add_sync(kAll, x.a & 0xffffu), __reduce_add_sync(kAll, x.a >> 16),
                      __reduce_add_sync(kAll, x.b & 0xffffu), __reduce_add_sync(kAll, x.b >> 16)};
  __syncthreads();                         // (the warps' sums of the scan before are read)
  if (lane == 31) {
    s_warp[warp] = mine;
    s_warp[warp].a = sum.a, s_warp[warp].b = sum.b;
  }
  __syncthreads();
  const WarpSums w = lane < warps ? s_warp[lane] : WarpSums{0, 0, 0, 0, 0, 0};
  const Two all = inclusive(Two{w.a, w.b});
  const unsigned a0 = __shfl_sync(kAll, all.a, warp > 0 ? warp - 1 : 0);
  const unsigned b0 = __shfl_sync(kAll, all.b, warp > 0 ? warp - 1 : 0);
  totals->a = ((unsigned long long)__reduce_add_sync(kAll, w.a_high) << 16) + __reduce_add_sync(kAll, w.a_low);
  totals->b = ((unsigned long long)__reduce_add_sync(kAll, w.b_high) << 16) + __reduce_add_sync(kAll, w.b_low);
  return Two{(warp > 0 ? a0 : 0) + sum.a - x.a, (warp > 0 ? b0 : 0) + sum.b - x.b};
}

// What request b adds (tokens, pages) or gives back (pages); false: out of range.
__device__ __forceinline__ bool request(const GdnPoolArgs& p, const GdnPlanArgs& a, int b,
                                        const Shared& s, Two* out) {
  const int row = a.rows ? a.rows[b] : b;
  const int len = a.len[b], more = a.more ? a.more[b] : 0;
  const int mask = (1 << p.page_shift) - 1;
  s.row[b] = row < 0 ? -1 : row;
  s.held[b] = s.from[b] = 0;
  *out = Two{0, 0};
  if (row < 0) return true;
  if (row >= p.num_rows || len < 0 || more < 0) return false;
  const int held = p.held[row];
  if (held < 0 || held > p.max_pages) return false;
  s.held[b] = held;
  const long long after = (long long)len + more;
  const long long pages = (after + mask) >> p.page_shift;
  if (a.more) {                            // a plan
    if (pages > p.max_pages) return false;
    s.from[b] = len;
    *out = Two{(unsigned)more, pages > held ? (unsigned)(pages - held) : 0u};
  } else {
    s.from[b] = (int)(pages < held ? pages : held);
    *out = Two{0, (unsigned)(held - s.from[b])};
  }
  return true;
}

// Fills s; false (in every thread): some request is out of range.
__device__ __forceinline__ bool scan_requests(const GdnPoolArgs& p, const GdnPlanArgs& a,
                                              const Shared& s, Totals* totals) {
  Totals sum{0, 0};
  bool good = true;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    Two x{0, 0};
    Totals block;
    if (b < a.B) good = request(p, a, b, s, &x) && good;
    const Two before = scan(x, &block);
    if (b < a.B) {
      s.tokens[b] = (int)((unsigned)sum.a + before.a);
      s.pages[b] = (int)((unsigned)sum.b + before.b);
    }
    sum.a += block.a;
    sum.b += block.b;
  }
  if (threadIdx.x == 0) {
    s.tokens[a.B] = (int)sum.a;
    s.pages[a.B] = (int)sum.b;
  }
  *totals = sum;
  return !__syncthreads_or(!good);
}

// The request that packed token t belongs to: the last whose first token is at or before it.
__device__ __forceinline__ int request_of(const Shared& s, int B, int t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.tokens[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// How block tables are shared out: `lanes` neighbours (a power of two) take a request's entries,
// kAtOnce each at a time, so that short tables leave no warp waiting for one request after the other
// (a plan and a release of 151 requests of one page 14.6 us with a warp each).
struct Tables {
  int lanes, lane, columns, pieces;        // of a request's table: entries at a time, and how often
  int first, step;                         // of the pieces: this lane's first, and the next
};
__device__ __forceinline__ Tables share_tables(int max_pages, int tid, int threads) {
  const int needed = (max_pages + kAtOnce - 1) / kAtOnce;
  const int shift = needed <= 1 ? 0 : min(5, 32 - __clz(needed - 1));
  const int columns = kAtOnce << shift;
  return Tables{1 << shift, tid & ((1 << shift) - 1), columns, (max_pages + columns - 1) / columns,
                tid >> shift, threads >> shift};
}

// The pool's and the requests' state after a plan.
__device__ __forceinline__ void write_state(const GdnPoolArgs& p, const GdnPlanArgs& a,
                                            const Shared& s, int left, int tid, int threads) {
  for (int b = tid; b < a.B; b += threads) {
    const int row = s.row[b], need = s.pages[b + 1] - s.pages[b];
    if (need > 0 && in_bounds(&g_err_kv, row >= 0 && row < p.num_rows))
      p.held[row] = s.held[b] + need;
    if (a.len_out)
      a.len_out[b] = row < 0 ? -1 : s.from[b] + s.tokens[b + 1] - s.tokens[b];
  }
  if (a.cu_seqlens)
    for (int b = tid; b <= a.B; b += threads) a.cu_seqlens[b] = s.tokens[b];
  if (tid == 0) *p.free_count = left;
}

// What a launch of the plan does: all of it (one cluster), or its two halves, the outputs by many
// CTAs, then the pool's new state by one, which reads everything before it waits for the other.
enum { kAll = 0, kOutputs = 1, kState = 2 };

template <int kPart>
__global__ void __launch_bounds__(kMostThreads) gdn_page_plan_kernel(GdnPoolArgs p, GdnPlanArgs a) {
  extern __shared__ int smem[];
  const Shared s = carve(smem, a.B);
  const int rank = kPart == kAll ? cluster_rank() : blockIdx.x;
  const int ctas = kPart == kAll ? cluster_size() : gridDim.x;
  const int tid = rank * blockDim.x + threadIdx.x, threads = ctas * blockDim.x;
  // Nothing is read before everything earlier is done; the second half of a large plan, which may
  // start from here on, reads the pool beside the first.
  if (kPart != kState) pdl_wait();
  pdl_trigger();
  const int count = *p.free_count, fill = a.slots || a.positions ? a.capacity : 0;
  Totals totals;
  bool good = scan_requests(p, a, s, &totals);
  good = good && count >= 0 && count <= p.num_pages && totals.a <= (unsigned long long)a.capacity &&
         totals.b <= (unsigned long long)count;
  // every CTA has read the pool's state and the lengths before they change
  if (kPart == kAll) cluster_sync();
  if (kPart == kState) pdl_wait();
  if (!good) {                             // nothing is given
    if (kPart != kOutputs && tid == 0) atomicOr(&g_err_kv, kErrIndex);
    if (kPart != kState)
      for (long long t = tid; t < fill; t += threads) {
        if (a.slots) a.slots[t] = -1;
        if (a.positions) a.positions[t] = 0;
      }
    if (kPart != kOutputs && a.cu_seqlens)
      for (int b = tid; b <= a.B; b += threads) a.cu_seqlens[b] = 0;
    return;
  }
  // ---- the requests' new state
  if (kPart != kOutputs) write_state(p, a, s, count - (int)totals.b, tid, threads);
  if (kPart == kState) return;
  // ---- block tables
  const int lane = threadIdx.x & 31, warps = threads >> 5;
  const Tables l = share_tables(p.max_pages, tid, threads);
  for (long long w = l.first; w < (long long)a.B * l.pieces; w += l.step) {
    const int b = (int)(w / l.pieces), c0 = (int)(w - (long long)b * l.pieces) * l.columns;
    const int row = s.row[b], held = s.held[b], first = s.pages[b];
    const int end = min(c0 + l.columns, held + s.pages[b + 1] - first);
    if (row < 0) continue;
    int* table = p.table + (long long)row * p.max_pages;
    int* pages = a.pages ? a.pages + (long long)b * p.max_pages : nullptr;
    int page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int c = c0 + k * l.lanes + l.lane;
      page[k] = 0;
      if (c < end && (pages || c >= held) && in_bounds(&g_err_kv, c >= 0 && c < p.max_pages))
        page[k] = c >= held ? p.free_pages[count - 1 - (first + c - held)] : table[c];
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int c = c0 + k * l.lanes + l.lane;
      if (c >= end || !in_bounds(&g_err_kv, c >= 0 && c < p.max_pages)) continue;
      if (c >= held) table[c] = page[k];
      if (pages) pages[c] = page[k];
    }
  }
  // ---- the tokens, a warp up to kInRow times 32 in a row, as many as there are for it (a lane looks
  // its request up once, as long as its next token belongs to it too)
  const int total = (int)totals.a, mask = (1 << p.page_shift) - 1;
  const int in_row = fill <= threads ? 1 : fill <= 2 * threads ? 2 : kInRow;
  for (long long t1 = (long long)(tid >> 5) * (32 * in_row); t1 < fill; t1 += (long long)warps * (32 * in_row)) {
    const int* table = nullptr;            // of the lane's request
    const int* fresh = nullptr;            // its new pages, from the end
    int until = 0, back = 0, held = 0;     // where its tokens end, and what is taken off a packed token
    int at[kInRow], page[kInRow];
#pragma unroll
    for (int k = 0; k < kInRow; ++k) {
      const long long t = t1 + k * 32 + lane;
      page[k] = at[k] = -1;
      if (k >= in_row || t >= total) continue;
      if (t >= until) {
        const int b = request_of(s, a.B, (int)t), row = s.row[b];
        until = s.tokens[b + 1], back = s.tokens[b] - s.from[b], held = s.held[b];
        table = p.table + (long long)row * p.max_pages;
        fresh = p.free_pages + (count - 1 - s.pages[b] + held);
      }
      at[k] = (int)t - back;
      const int c = at[k] >> p.page_shift;
      if (a.slots && in_bounds(&g_err_kv, c >= 0 && c < p.max_pages)) page[k] = c < held ? table[c] : fresh[-c];
    }
#pragma unroll
    for (int k = 0; k < kInRow; ++k) {
      const long long t = t1 + k * 32 + lane;
      if (k >= in_row || t >= fill) continue;
      const bool some = page[k] >= 0 && page[k] < p.num_pages;
      if (a.slots && t < total && !some) atomicOr(&g_err_kv, kErrIndex);
      if (a.slots) a.slots[t] = some ? (page[k] << p.page_shift) + (at[k] & mask) : -1;
      if (a.positions) a.positions[t] = at[k] >= 0 ? a.offset + at[k] : 0;
    }
  }
}

__global__ void __launch_bounds__(kMostThreads) gdn_page_release_kernel(GdnPoolArgs p, GdnPlanArgs a) {
  extern __shared__ int smem[];
  const Shared s = carve(smem, a.B);
  const int rank = cluster_rank(), ctas = cluster_size();
  const int tid = rank * blockDim.x + threadIdx.x, threads = ctas * blockDim.x;
  pdl_wait();
  pdl_trigger();
  const int count = *p.free_count;
  Totals totals;
  bool good = scan_requests(p, a, s, &totals);
  good = good && count >= 0 && totals.b + (unsigned long long)count <= (unsigned long long)p.num_pages;
  cluster_sync();
  if (!good) {
    if (tid == 0) atomicOr(&g_err_kv, kErrIndex);
    return;
  }
  const int end = count + (int)totals.b;
  for (int b = tid; b < a.B; b += threads)
    if (s.pages[b + 1] > s.pages[b] &&
        in_bounds(&g_err_kv, s.row[b] >= 0 && s.row[b] < p.num_rows))
      p.held[s.row[b]] = s.from[b];
  if (tid == 0) *p.free_count = end;
  const Tables l = share_tables(p.max_pages, tid, threads);
  for (long long w = l.first; w < (long long)a.B * l.pieces; w += l.step) {
    const int b = (int)(w / l.pieces), c0 = (int)(w - (long long)b * l.pieces) * l.columns;
    const int first = s.pages[b], given = s.pages[b + 1] - first, kept = s.from[b];
    if (given == 0) continue;
    const int* table = p.table + (long long)s.row[b] * p.max_pages + kept;
    int page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int c = c0 + k * l.lanes + l.lane;
      page[k] = c < given && in_bounds(&g_err_kv, kept + c < p.max_pages) ? table[c] : 0;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int c = c0 + k * l.lanes + l.lane, to = end - 1 - (first + c);
      if (c < given && in_bounds(&g_err_kv, to >= count && to < p.num_pages)) p.free_pages[to] = page[k];
    }
  }
}

// The cluster for `words` of output: first more CTAs, then more threads, so that each thread has a
// few words.
template <typename K>
cudaError_t launch(K kernel, const GdnPoolArgs& p, const GdnPlanArgs& a, long long words,
                   unsigned* done, cudaStream_t stream) {
  int threads = 256, ctas = 1;
  while (ctas < kMaxCtas && words > (long long)ctas * threads * 2) ctas *= 2;
  while (threads < kMostThreads && words > (long long)ctas * threads * 4) threads *= 2;
  const size_t smem = shared_bytes(a.B);
  if (smem > kUnasked) {
    const cudaError_t e = set_smem_once(kernel, (int)shared_bytes(kGdnMaxRequests), done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, a);
}

}  // namespace pages
}  // namespace

cudaError_t gdn_launch_page_plan(const GdnPoolArgs& p, const GdnPlanArgs& a, cudaStream_t stream) {
  static unsigned done[3] = {};
  const long long fill = a.slots || a.positions ? a.capacity : 0;
  const long long words = std::max(fill, (long long)a.B * p.max_pages);
  if (words <= pages::kOneCluster)
    return pages::launch(pages::gdn_page_plan_kernel<pages::kAll>, p, a, words, &done[0], stream);
  const size_t smem = pages::shared_bytes(a.B);
  if (smem > pages::kUnasked) {
    const int most = (int)pages::shared_bytes(kGdnMaxRequests);
    cudaError_t e = set_smem_once(pages::gdn_page_plan_kernel<pages::kOutputs>, most, &done[1]);
    if (e == cudaSuccess) e = set_smem_once(pages::gdn_page_plan_kernel<pages::kState>, most, &done[2]);
    if (e != cudaSuccess) return e;
  }
  const unsigned ctas = (unsigned)std::min(152ll, (words + 2047) / 2048);
  const cudaError_t e = launch_pdl(true, pages::gdn_page_plan_kernel<pages::kOutputs>, dim3(ctas),
                                   dim3(512), smem, stream, p, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(true, pages::gdn_page_plan_kernel<pages::kState>, dim3(1), dim3(512), smem, stream,
                    p, a);
}

cudaError_t gdn_launch_page_release(const GdnPoolArgs& p, const GdnPlanArgs& a,
                                    cudaStream_t stream) {
  static unsigned done = 0;
  return pages::launch(pages::gdn_page_release_kernel, p, a, (long long)a.B * p.max_pages, &done, stream);
}
