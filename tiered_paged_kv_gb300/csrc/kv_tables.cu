// Page tables and slot maps from request lengths.
//
// With have = ceil(old / 64) and want = ceil(new / 64), three running sums over the
// requests settle everything: new tokens (where a request's tokens begin), pages given
// back, and pages taken.  The free stack after the releases is the old stack followed by
// the pages given back in order, and the i-th page taken in all is its (there - 1 - i)-th
// entry, so every page finds its slot by itself: one thread a page, wherever it belongs.
// A pushed page that is taken again is looked up in the giver's table row, which this
// call only reads.
//
// One block makes the sums and the new pages and writes the requests' results, all of
// its inputs read before (lengths and the free count may be updated in place).  The maps
// of the tokens follow from those results and the tables: up to kOneBlock tokens in the
// same block; more in a second launch over the whole device, whose start overlaps the
// first.  Bound: latency; the maps are 16 bytes per token.  Measured: 64 requests of one new
// token 3.9 us, 1,000 requests with 63 thousand new tokens 11.5 us (of them 7.5 in the
// first block).
#include "paged.cuh"

namespace tpk {

constexpr int kTabThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillTokens = 4;  // of a thread, their lookups in flight together
// Tokens that the block fills in itself: 2,100 tokens of 64 requests take 6.3 us in one
// block and 6.9 with the second launch, 4,200 take 7.3 and 6.8, 33,000 take 25 and 7.3.
constexpr int kOneBlock = 2048;

// Exclusive prefix sums of two values over the block's threads; total: the sums of all.
__device__ __forceinline__ void block_scan(ulonglong2& v, ulonglong2* warp_sums, ulonglong2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto inclusive = [&](ulonglong2 x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long a = __shfl_up_sync(0xffffffffu, x.x, d), b = __shfl_up_sync(0xffffffffu, x.y, d);
      if (lane >= d) {
        x.x += a;
        x.y += b;
      }
    }
    return x;
  };
  const ulonglong2 inc = inclusive(v);
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  const ulonglong2 mine = warp_sums[lane], w = inclusive(mine);
  total.x = __shfl_sync(0xffffffffu, w.x, 31);
  total.y = __shfl_sync(0xffffffffu, w.y, 31);
  v.x = __shfl_sync(0xffffffffu, w.x - mine.x, warp) + inc.x - v.x;
  v.y = __shfl_sync(0xffffffffu, w.y - mine.y, warp) + inc.y - v.y;
}

// For each u the last index i in [0, n) with a[i] <= x[u] (a ascending, a[0] <= x[u]); the
// same number of steps for all, so that their loads are in flight together.
template <int N>
__device__ __forceinline__ void last_not_above(const int32_t* a, int n, const int (&x)[N], int (&out)[N]) {
#pragma unroll
  for (int u = 0; u < N; ++u) out[u] = 0;
  for (int step = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; step > 0; step >>= 1)
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (out[u] + step < n && a[out[u] + step] <= x[u]) out[u] += step;
}

__device__ __forceinline__ int pages_of(int tokens) { return (int)(((int64_t)tokens + 63) >> 6); }

// The maps of tokens t, t + step, ... (kFillTokens of them), from the requests' results.
__device__ __forceinline__ void fill_maps(const TablesParams& p, const int32_t* off, int t, int step) {
  const int n = p.n_req, tokens = off[n];
  int b[kFillTokens], len[kFillTokens], ok[kFillTokens], pos[kFillTokens], s[kFillTokens];
#pragma unroll
  for (int u = 0; u < kFillTokens; ++u) pos[u] = t + u * step;
  last_not_above(off, n, pos, b);
#pragma unroll
  for (int u = 0; u < kFillTokens; ++u)
    if (pos[u] >= tokens) b[u] = -1;
#pragma unroll
  for (int u = 0; u < kFillTokens; ++u) {
    len[u] = b[u] >= 0 ? p.len_out[b[u]] : 0;
    ok[u] = b[u] >= 0 ? p.granted[b[u]] : 0;
  }
#pragma unroll
  for (int u = 0; u < kFillTokens; ++u) {
    pos[u] = 0;
    s[u] = -1;
    if (b[u] < 0) continue;
    const int begin = off[b[u]], count = off[b[u] + 1] - begin;
    pos[u] = len[u] - (ok[u] ? count : 0) + (t + u * step - begin);
    if (ok[u]) s[u] = p.page_table[(int64_t)b[u] * p.max_pages + (pos[u] >> 6)];
  }
#pragma unroll
  for (int u = 0; u < kFillTokens; ++u) {
    const int i = t + u * step;
    if (i >= p.max_tokens) break;
    p.slot_map[i] = ok[u] ? (int64_t)s[u] * kPageTokens + (pos[u] & 63) : -1;
    p.positions[i] = pos[u];
    p.token_req[i] = b[u];
  }
}

template <int N>
struct Some {
  static constexpr int value = N;
};

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p, int fill) {
  extern __shared__ int32_t sm[];
  __shared__ ulonglong2 warp_sums[32];
  __shared__ int taken_all;
  const int n = p.n_req, tid = threadIdx.x;
  int32_t* off = sm;             // [n + 1] where the request's new tokens begin
  int32_t* taken = off + n + 1;  // [n] pages taken before it
  int32_t* gave = taken + n;     // [n] pages given back before it
  uint8_t* fine = reinterpret_cast<uint8_t*>(gave + n);  // [n] granted
  wait_before();
  start_next();

  const int each = (n + kTabThreads - 1) / kTabThreads;
  const int b0 = min(tid * each, n), b1 = min(b0 + each, n);
  const int n_free = min(max(*p.n_free_in, 0), p.free_cap);
  if (tid == 0) taken_all = 0;

  // new tokens; pages taken (high half) and given back (low half), whose sums stay below
  // 2^31 because every request counted fits its table row and n_req * max_pages < 2^31
  const uint64_t cap = (uint64_t)p.max_tokens;
  auto pages_fit = [&](int a, int c) {
    return a >= 0 && c >= 0 && pages_of(a) <= p.max_pages && pages_of(c) <= p.max_pages;
  };
  auto packed = [](int d) { return d > 0 ? (uint64_t)d << 32 : (uint64_t)(uint32_t)(-d); };
  ulonglong2 run = make_ulonglong2(0, 0), total;
  for (int b = b0; b < b1; ++b) {
    const int a = p.len_old[b], c = p.len_new[b];
    if (a >= 0 && c > a) run.x += (uint32_t)(c - a);
    const bool fits = pages_fit(a, c);
    const int d = fits ? pages_of(c) - pages_of(a) : 0;
    fine[b] = fits;
    taken[b] = d;
    run.y += packed(d);
  }
  block_scan(run, warp_sums, total);
  if (tid == 0) off[n] = (int)min((uint64_t)total.x, cap);
  uint64_t at = run.x;
  for (int b = b0; b < b1; ++b) {
    const int a = p.len_old[b], c = p.len_new[b];
    off[b] = (int)min(at, cap);
    if (a >= 0 && c > a) {
      at += (uint32_t)(c - a);
      if (at > cap) {  // no place in the maps: it takes no pages either
        fine[b] = 0;
        taken[b] = 0;
      }
    }
  }
  if (total.x > cap) {  // then the pages are summed again without those requests
    run = make_ulonglong2(0, 0);
    for (int b = b0; b < b1; ++b) run.y += packed(taken[b]);
    block_scan(run, warp_sums, total);
  }
  const int there = n_free + (int)(uint32_t)total.y;  // the stack's height after the releases
  int last = 0;
  for (int b = b0; b < b1; ++b) {
    const int d = taken[b];
    taken[b] = (int)(run.y >> 32);
    gave[b] = (int)(uint32_t)run.y;
    run.y += packed(d);
    if (d > 0) {
      const int after = (int)(run.y >> 32);
      if (after <= there) last = after; else fine[b] = 0;
    }
  }
  if (last > 0) atomicMax(&taken_all, last);
  __syncthreads();

  const int left = there - taken_all;  // the stack's height at the end
  // the r-th page given back is row entry r - gave[b] past those that its giver keeps
  auto pushed = [&](int b, int r) {
    return p.page_table[(int64_t)b * p.max_pages + pages_of(p.len_new[b]) + (r - gave[b])];
  };
  // both lists, several entries a thread at a time where there are many: their lookups
  // are in flight together
  const int keep = min(left, p.free_cap);
  auto keep_some = [&](int i0, auto some) {
    constexpr int N = decltype(some)::value;
    int r[N], b[N], s[N];
#pragma unroll
    for (int u = 0; u < N; ++u) r[u] = i0 + u * kTabThreads - n_free;
    last_not_above(gave, n, r, b);
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (i0 + u * kTabThreads < keep) s[u] = pushed(b[u], r[u]);
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (i0 + u * kTabThreads < keep) p.free_slots[i0 + u * kTabThreads] = s[u];
  };
  auto take_some = [&](int i0, auto some) {
    constexpr int N = decltype(some)::value;
    int i[N], r[N], b[N], from[N], s[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      i[u] = i0 + u * kTabThreads;
      r[u] = there - 1 - i[u] - n_free;
    }
    last_not_above(taken, n, i, b);
    if (r[0] >= 0) last_not_above(gave, n, r, from);
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (i[u] < taken_all) s[u] = r[u] < 0 ? p.free_slots[there - 1 - i[u]] : pushed(from[u], r[u]);
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (i[u] < taken_all && fine[b[u]])
        p.page_table[(int64_t)b[u] * p.max_pages + pages_of(p.len_old[b[u]]) + (i[u] - taken[b[u]])] = s[u];
  };
  if (keep - n_free > kTabThreads)
    for (int i = n_free + tid; i < keep; i += 4 * kTabThreads) keep_some(i, Some<4>{});
  else
    for (int i = n_free + tid; i < keep; i += kTabThreads) keep_some(i, Some<1>{});
  if (tid == 0 && left > p.free_cap) atomicOr(p.status, kStatusBadSlot);
  if (taken_all > kTabThreads)
    for (int i = tid; i < taken_all; i += 4 * kTabThreads) take_some(i, Some<4>{});
  else
    for (int i = tid; i < taken_all; i += kTabThreads) take_some(i, Some<1>{});

  __syncthreads();  // the lengths and the free count have been read
  if (tid == 0) *p.n_free_out = min(left, p.free_cap);
  for (int b = tid; b <= n; b += kTabThreads) p.tok_off[b] = off[b];
  for (int b = tid; b < n; b += kTabThreads) {
    const int a = p.len_old[b], c = p.len_new[b];
    p.granted[b] = fine[b];
    p.len_out[b] = fine[b] ? c : a;
  }
  if (!fill) return;
  __syncthreads();
  for (int t = tid; t < p.max_tokens; t += kFillTokens * kTabThreads) fill_maps(p, off, t, kTabThreads);
}

__global__ void __launch_bounds__(kFillThreads) maps_kernel(const TablesParams p) {
  extern __shared__ int32_t off[];  // [n + 1]
  wait_before();
  for (int b = threadIdx.x; b <= p.n_req; b += kFillThreads) off[b] = p.tok_off[b];
  __syncthreads();
  fill_maps(p, off, blockIdx.x * (kFillThreads * kFillTokens) + threadIdx.x, kFillThreads);
}

cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream) {
  static DeviceOnce once;
  const int most = (3 * kMaxPagedReq + 1) * (int)sizeof(int32_t) + kMaxPagedReq;
  cudaError_t e = once.run(
      [&] { return cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most); });
  if (e != cudaSuccess) return e;
  const bool one = p.max_tokens <= kOneBlock;
  e = launch_early(tables_kernel, 1, kTabThreads, (3 * p.n_req + 1) * sizeof(int32_t) + p.n_req, stream, p, (int)one);
  if (e != cudaSuccess || one) return e;
  const int per_block = kFillThreads * kFillTokens;
  return launch_early(maps_kernel, (p.max_tokens + per_block - 1) / per_block, kFillThreads, (p.n_req + 1) * sizeof(int32_t),
                      stream, p);
}

}  // namespace tpk
