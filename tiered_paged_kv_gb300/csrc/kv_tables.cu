// Page tables and slot maps from request lengths.
//
// With have = ceil(old / 64) and want = ceil(new / 64), three running sums over the
// requests settle everything: new tokens (where a request's tokens begin), pages
// given back, and pages taken.  The free stack after the releases is the old stack
// followed by the pages given back in order, and the i-th page taken in all is its
// (there - 1 - i)-th entry, so any token finds its page without waiting for another:
// a page below `have` is in the table already, a later one is an entry of the stack,
// and the token at a page's first row also writes the table.  A pushed page that is
// taken again is looked up in the giver's table row, which this call only reads.
//
// Bound: latency (16 bytes per token written; the sums take two block-wide scans).
// Every block of one cluster makes the same scans and fills its share of the tokens;
// the lengths and the free count may be updated in place, so they are written after
// the cluster's barrier, when no block reads them any more.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace tpk {

constexpr int kTabThreads = 1024;

// Exclusive prefix sum over the block's threads; *total is the sum of all.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_sums, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  uint64_t before = 0, all = 0;
  const uint64_t mine = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
  uint64_t w = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += up;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  before = __shfl_sync(0xffffffffu, w - mine, warp);
  *total = all;
  return before + inc - v;
}

// The last index i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int32_t* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(int tokens) { return (int)(((int64_t)tokens + 63) >> 6); }

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ int32_t sm[];
  __shared__ uint64_t warp_sums[32];
  __shared__ int taken_all;
  const int n = p.n_req, tid = threadIdx.x;
  int32_t* off = sm;              // [n + 1] where the request's new tokens begin
  int32_t* taken = off + n + 1;   // [n] pages taken before it; ~ that if it is refused
  int32_t* gave = taken + n;      // [n] pages given back before it
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();

  const int each = (n + kTabThreads - 1) / kTabThreads;
  const int b0 = min(tid * each, n), b1 = min(b0 + each, n);
  const int n_free = min(max(*p.n_free_in, 0), p.free_cap);
  if (tid == 0) taken_all = 0;

  uint64_t sum = 0, total;
  for (int b = b0; b < b1; ++b) {
    const int a = p.len_old[b], c = p.len_new[b];
    if (a >= 0 && c > a) sum += (uint32_t)(c - a);
  }
  uint64_t at = block_scan(sum, warp_sums, &total);
  const uint64_t cap = (uint64_t)p.max_tokens;
  if (tid == 0) off[n] = (int)min(total, cap);
  // pages taken (high half) and given back (low half); both sums stay below 2^31
  // because every request counted fits its table row and n_req * max_pages < 2^31
  uint64_t pages = 0;
  for (int b = b0; b < b1; ++b) {
    const int a = p.len_old[b], c = p.len_new[b];
    off[b] = (int)min(at, cap);
    if (a >= 0 && c > a) at += (uint32_t)(c - a);
    const bool fits = a >= 0 && c >= 0 && pages_of(a) <= p.max_pages && pages_of(c) <= p.max_pages &&
                      (c <= a || at <= cap);
    const int d = fits ? pages_of(c) - pages_of(a) : 0;
    taken[b] = fits ? d : 0x7fffffff;
    pages += d > 0 ? (uint64_t)d << 32 : (uint64_t)(uint32_t)(-d);
  }
  uint64_t run = block_scan(pages, warp_sums, &total);
  const int there = n_free + (int)(uint32_t)total;  // the stack's height after the releases
  int last = 0;
  for (int b = b0; b < b1; ++b) {
    const int d = taken[b];
    const bool fits = d != 0x7fffffff;
    const int before = (int)(run >> 32);
    gave[b] = (int)(uint32_t)run;
    bool ok = fits;
    if (fits) {
      run += d > 0 ? (uint64_t)d << 32 : (uint64_t)(uint32_t)(-d);
      if (d > 0) {
        ok = (int)(run >> 32) <= there;
        if (ok) last = (int)(run >> 32);
      }
    }
    taken[b] = ok ? before : ~before;
  }
  if (last > 0) atomicMax(&taken_all, last);
  __syncthreads();

  const int left = there - taken_all;  // the stack's height at the end
  auto pushed = [&](int r) {           // the r-th page given back
    const int b = last_not_above(gave, n, r);
    return p.page_table[(int64_t)b * p.max_pages + pages_of(p.len_new[b]) + (r - gave[b])];
  };
  const int me = rank * kTabThreads + tid, step = ranks * kTabThreads;
  for (int i = n_free + me; i < min(left, p.free_cap); i += step) p.free_slots[i] = pushed(i - n_free);
  if (me == 0 && left > p.free_cap) atomicOr(p.status, kStatusBadSlot);

  const int tokens = off[n];
  for (int t = me; t < p.max_tokens; t += step) {
    int64_t slot = -1;
    int pos = 0, b = -1;
    if (t < tokens) {
      b = last_not_above(off, n, t);
      const int a = p.len_old[b];
      pos = a + (t - off[b]);
      const int before = taken[b];
      if (before >= 0) {
        const int page = pos >> 6, have = pages_of(a);
        int32_t* entry = p.page_table + (int64_t)b * p.max_pages + page;
        int s;
        if (page < have) {
          s = *entry;
        } else {
          const int i = there - 1 - (before + page - have);
          s = i < n_free ? p.free_slots[i] : pushed(i - n_free);
          if ((pos & 63) == 0) *entry = s;
        }
        slot = (int64_t)s * kPageTokens + (pos & 63);
      }
    }
    p.slot_map[t] = slot;
    p.positions[t] = pos;
    p.token_req[t] = b;
  }

  if (ranks > 1) cluster.sync(); else __syncthreads();
  if (rank != 0) return;
  if (tid == 0) *p.n_free_out = min(left, p.free_cap);
  for (int b = tid; b <= n; b += kTabThreads) p.tok_off[b] = off[b];
  for (int b = tid; b < n; b += kTabThreads) {
    const bool ok = taken[b] >= 0;
    const int a = p.len_old[b], c = p.len_new[b];
    p.granted[b] = ok;
    p.len_out[b] = ok ? c : a;
  }
}

// Blocks of the cluster: one fills up to 2048 tokens (two per thread); past that the
// fill is longer than the cluster's barrier, and eight (the portable size) share it.
cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream) {
  static DeviceOnce once;
  const int most = (3 * kMaxPagedReq + 1) * (int)sizeof(int32_t);
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  const int blocks = p.max_tokens <= 2048 ? 1 : 8;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kTabThreads);
  cfg.dynamicSmemBytes = (size_t)(3 * p.n_req + 1) * sizeof(int32_t);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tables_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tpk
