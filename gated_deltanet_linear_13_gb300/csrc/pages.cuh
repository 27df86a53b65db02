// Pages, slots and positions of a step's new tokens, and pages given back, from the requests'
// lengths on the device.
//
// Both calls are a scan over the B requests (tokens and pages that each adds or gives back), a few
// words a token or table entry behind it, and the new state of the pool.  The scan is a few
// hundred nanoseconds, so every CTA of one cluster does it for itself and takes its share of the
// rest; a cluster barrier between the last read of the pool's counts and their update is all the
// order that is needed, so a call is one launch and keeps nothing between calls.
// Part of kv_cache.cu, whose error word it uses.
#pragma once

#include <algorithm>

#include "common.cuh"

using namespace gdn;

namespace {
namespace pages {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;                // of the cluster (the portable most)
constexpr int kColumns = 128;              // of a block table a warp takes at a time

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

// Sums of two numbers over the threads before this one; *totals gets the block's.
struct Two {
  unsigned long long a, b;
};
__device__ __forceinline__ Two scan(Two x, Two* totals) {
  __shared__ Two s_warp[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Two sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long a = __shfl_up_sync(0xffffffffu, sum.a, o);
    const unsigned long long b = __shfl_up_sync(0xffffffffu, sum.b, o);
    if (lane >= o) sum.a += a, sum.b += b;
  }
  __syncthreads();                         // (the warps' sums of the scan before are read)
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  Two before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const Two t = s_warp[w];
    if (w < warp) before.a += t.a, before.b += t.b;
    all.a += t.a, all.b += t.b;
  }
  *totals = all;
  return Two{before.a + sum.a - x.a, before.b + sum.b - x.b};
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
    *out = Two{(unsigned long long)more, pages > held ? (unsigned long long)(pages - held) : 0};
  } else {
    s.from[b] = (int)(pages < held ? pages : held);
    *out = Two{0, (unsigned long long)(held - s.from[b])};
  }
  return true;
}

// Fills s; false (in every thread): some request is out of range.
__device__ __forceinline__ bool scan_requests(const GdnPoolArgs& p, const GdnPlanArgs& a,
                                              const Shared& s, Two* totals) {
  Two sum{0, 0};
  bool good = true;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    Two x{0, 0}, block;
    if (b < a.B) good = request(p, a, b, s, &x) && good;
    const Two before = scan(x, &block);
    if (b < a.B) {
      s.tokens[b] = (int)(sum.a + before.a);
      s.pages[b] = (int)(sum.b + before.b);
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

__global__ void __launch_bounds__(kThreads) gdn_page_plan_kernel(GdnPoolArgs p, GdnPlanArgs a) {
  extern __shared__ int smem[];
  const Shared s = carve(smem, a.B);
  const int rank = cluster_rank(), ctas = cluster_size();
  const int tid = rank * kThreads + threadIdx.x, threads = ctas * kThreads;
  const int count = *p.free_count, fill = a.slots || a.positions ? a.capacity : 0;
  Two totals;
  bool good = scan_requests(p, a, s, &totals);
  good = good && count >= 0 && count <= p.num_pages && totals.a <= (unsigned long long)a.capacity &&
         totals.b <= (unsigned long long)count;
  cluster_sync();                          // every CTA has read the pool's state and the lengths
  if (!good) {                             // nothing is given
    if (tid == 0) atomicOr(&g_err_kv, kErrIndex);
    for (int t = tid; t < fill; t += threads) {
      if (a.slots) a.slots[t] = -1;
      if (a.positions) a.positions[t] = 0;
    }
    if (a.cu_seqlens)
      for (int b = tid; b <= a.B; b += threads) a.cu_seqlens[b] = 0;
    return;
  }
  // ---- the requests' new state
  for (int b = tid; b < a.B; b += threads) {
    const int row = s.row[b], need = s.pages[b + 1] - s.pages[b];
    if (need > 0 && in_bounds(&g_err_kv, row >= 0 && row < p.num_rows))
      p.held[row] = s.held[b] + need;
    if (a.len_out)
      a.len_out[b] = row < 0 ? -1 : s.from[b] + s.tokens[b + 1] - s.tokens[b];
  }
  if (a.cu_seqlens)
    for (int b = tid; b <= a.B; b += threads) a.cu_seqlens[b] = s.tokens[b];
  if (tid == 0) *p.free_count = count - (int)totals.b;
  // ---- block tables: a warp kColumns of a request's pages at a time
  const int lane = threadIdx.x & 31, warps = ctas * kWarps;
  const int pieces = (p.max_pages + kColumns - 1) / kColumns;
  for (long long w = tid >> 5; w < (long long)a.B * pieces; w += warps) {
    const int b = (int)(w / pieces), c0 = (int)(w - (long long)b * pieces) * kColumns;
    const int row = s.row[b], held = s.held[b], first = s.pages[b];
    const int end = min(c0 + kColumns, held + s.pages[b + 1] - first);
    if (row < 0) continue;
    int* table = p.table + (long long)row * p.max_pages;
    int* pages = a.pages ? a.pages + (long long)b * p.max_pages : nullptr;
    for (int c = (pages ? c0 : max(c0, held)) + lane; c < end; c += 32) {
      if (!in_bounds(&g_err_kv, c >= 0 && c < p.max_pages)) break;
      const bool fresh = c >= held;
      const int page = fresh ? p.free_pages[count - 1 - (first + c - held)] : table[c];
      if (fresh) table[c] = page;
      if (pages) pages[c] = page;
    }
  }
  // ---- the tokens
  const int total = (int)totals.a, mask = (1 << p.page_shift) - 1;
  for (int t = tid; t < fill; t += threads) {
    int slot = -1, position = 0;
    if (t < total) {
      const int b = request_of(s, a.B, t), at = s.from[b] + t - s.tokens[b];
      position = a.offset + at;
      if (a.slots) {
        const int c = at >> p.page_shift, held = s.held[b], row = s.row[b];
        int page = -1;
        if (in_bounds(&g_err_kv, row >= 0 && c < p.max_pages))
          page = c < held ? p.table[(long long)row * p.max_pages + c]
                          : p.free_pages[count - 1 - (s.pages[b] + c - held)];
        if (page >= 0 && page < p.num_pages) slot = (page << p.page_shift) + (at & mask);
        else atomicOr(&g_err_kv, kErrIndex);
      }
    }
    if (a.slots) a.slots[t] = slot;
    if (a.positions) a.positions[t] = position;
  }
}

__global__ void __launch_bounds__(kThreads) gdn_page_release_kernel(GdnPoolArgs p, GdnPlanArgs a) {
  extern __shared__ int smem[];
  const Shared s = carve(smem, a.B);
  const int rank = cluster_rank(), ctas = cluster_size();
  const int tid = rank * kThreads + threadIdx.x, threads = ctas * kThreads;
  const int count = *p.free_count;
  Two totals;
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
  const int lane = threadIdx.x & 31, warps = ctas * kWarps;
  const int pieces = (p.max_pages + kColumns - 1) / kColumns;
  for (long long w = tid >> 5; w < (long long)a.B * pieces; w += warps) {
    const int b = (int)(w / pieces), c0 = (int)(w - (long long)b * pieces) * kColumns;
    const int first = s.pages[b], given = s.pages[b + 1] - first, kept = s.from[b];
    if (given == 0) continue;
    const int* table = p.table + (long long)s.row[b] * p.max_pages + kept;
    for (int c = c0 + lane; c < min(c0 + kColumns, given); c += 32) {
      const int to = end - 1 - (first + c);
      if (in_bounds(&g_err_kv, to >= count && to < p.num_pages && kept + c < p.max_pages))
        p.free_pages[to] = table[c];
    }
  }
}

// CTAs of the cluster for `words` of output: one CTA's threads take a few words each before
// another CTA is worth its place.
template <typename K>
cudaError_t launch(K kernel, const GdnPoolArgs& p, const GdnPlanArgs& a, long long words,
                   unsigned* done, cudaStream_t stream) {
  int ctas = 1;
  while (ctas < kMaxCtas && words > (long long)ctas * kThreads * 2) ctas *= 2;
  const size_t smem = shared_bytes(a.B);
  if (smem > 48 * 1024) {
    const cudaError_t e = set_smem_once(kernel, (int)shared_bytes(kGdnMaxRequests), done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, a);
}

}  // namespace pages
}  // namespace

cudaError_t gdn_launch_page_plan(const GdnPoolArgs& p, const GdnPlanArgs& a, cudaStream_t stream) {
  static unsigned done = 0;
  const long long fill = a.slots || a.positions ? a.capacity : 0;
  const long long tables = (long long)a.B * p.max_pages;
  return pages::launch(pages::gdn_page_plan_kernel, p, a, std::max(fill, tables), &done, stream);
}

cudaError_t gdn_launch_page_release(const GdnPoolArgs& p, const GdnPlanArgs& a,
                                    cudaStream_t stream) {
  static unsigned done = 0;
  return pages::launch(pages::gdn_page_release_kernel, p, a, (long long)a.B * p.max_pages, &done, stream);
}
