// Upkeep of pages that several requests share: forks (with ends and cuts), compaction, and the
// copies that these ask for.
//
// Forks and compaction are bookkeeping on whole numbers: a few bytes for each page-table entry
// and each slot, in phases that each need all of the phase before.  A small pool and table go to one
// block, which keeps what it counts in shared memory (a beam step of 64 rows, 367 slots: 9.5 us
// as a cluster, 5.8 so; compaction of 900 slots 10.8 and 4.6; one_block).  Others go to one cluster of kParts
// blocks, whose barrier separates the phases: they are bound by the latency of their phases, not
// by what eight SMs can read, and a barrier of a cluster costs less than a launch.  Sums and counts
// go by integer atomics, which give the same in any order; ranks go by scans, so that the result
// is the one that the definition's order gives.
//
// Bound: latency for those two, HBM for the copies (two bytes moved for each byte of a page).
#include <climits>

#include "paged.cuh"

namespace tpk {

constexpr int kParts = 8;  // blocks of the cluster (as many as every device takes)
constexpr int kPartThreads = 1024;
constexpr int kPartWarps = kPartThreads / 32;
constexpr int kLocalSlots = 8192, kLocalEntries = 32768;  // of a pool, and of a table, that one block takes

// What differs between one block and a cluster.  Arrays that the threads share lie in shared memory,
// or in global memory, where what another block wrote must not come from this SM's L1.
template <bool kLocal>
struct Team {
  static constexpr int parts = kLocal ? 1 : kParts;
  // All threads have come here, and see what the others wrote before.
  static __device__ __forceinline__ void meet() {
    if (kLocal)
      __syncthreads();
    else
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  static __device__ __forceinline__ int get(const int32_t* p) { return kLocal ? *p : __ldcg(p); }
  static __device__ __forceinline__ int part() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return kLocal ? 0 : (int)r;
  }
};
__device__ __forceinline__ int pages_of(int tokens) { return (tokens >> 6) + ((tokens & 63) != 0); }

// How many of the block's threads below this one have the flag, and how many in all.
__device__ __forceinline__ int rank_in_block(bool flag, int* warp_counts, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned votes = __ballot_sync(0xffffffffu, flag);
  __syncthreads();  // the last call's counts have been read
  if (lane == 0) warp_counts[warp] = __popc(votes);
  __syncthreads();
  const int mine = warp_counts[lane];
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  total = __shfl_sync(0xffffffffu, inc, 31);
  return __shfl_sync(0xffffffffu, inc - mine, warp) + __popc(votes & ((1u << lane) - 1));
}

// The slots, cut into equal stretches for the parts; within a stretch tiles of a block's width.
struct Stretch {
  int begin, end;
  __device__ __forceinline__ Stretch(int n, int part, int parts) {
    const int per = (int)(((int64_t)n + parts - 1) / parts);
    begin = (int)min((int64_t)per * part, (int64_t)n);
    end = min(begin + per, n);
  }
};

// How many slots of the stretches before and behind this part's have the flag, and how many in all.
// For all threads; the parts meet in it.
template <bool kLocal, typename F>
__device__ __forceinline__ void count_flags(const Stretch& mine, int part, int* warp_counts, int32_t* counts, F flag, int& before,
                                            int& behind, int& all) {
  int count = 0;
  for (int i = mine.begin + (int)threadIdx.x; i < mine.end; i += kPartThreads) count += flag(i);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) count += __shfl_xor_sync(0xffffffffu, count, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_counts[threadIdx.x >> 5] = count;
  __syncthreads();
  int sum = warp_counts[threadIdx.x & 31];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  before = behind = 0;
  all = sum;
  if (kLocal) return;
  if (threadIdx.x == 0) counts[part] = sum;
  Team<kLocal>::meet();
  all = 0;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const int n = __ldcg(counts + i);
    all += n;
    if (i < part) before += n;
    if (i > part) behind += n;
  }
}

// ------------------------------------------------------------------- fork
// Holders: shares_in[x] + 1 hold slot x.  A request that changes (another source, or cut) lets its
// old pages go and takes up the whole pages that it keeps; base = holders after that.  A kept
// history that ends inside page x makes x the request's open page: it will be written on.
//   base = 0: the first of the requests with open page x keeps it, the others copy it;
//   base > 0: all of them copy it.
// A slot that is copied from is held by somebody, so that it is not handed out in the same call.
constexpr int kMostReq = kMaxPagedReq;
struct ForkShared {
  int counts[kPartWarps];
  int source[kMostReq];  // whose table row the request's pages come from
  int keep[kMostReq];    // tokens it keeps
  int page[kMostReq];    // its open page
  int fresh[kMostReq];   // the slot of its copied page; -1: none; -2: nothing to do, -3: refused
};
constexpr int kNone = -1, kSame = -2, kRefused = -3;

template <bool kLocal>
__global__ void __launch_bounds__(kPartThreads, 1) fork_kernel(const ForkParams p) {
  using Team = ::tpk::Team<kLocal>;
  extern __shared__ __align__(16) uint8_t raw[];
  ForkShared& S = *reinterpret_cast<ForkShared*>(raw);
  int32_t* const local = reinterpret_cast<int32_t*>(raw + sizeof(ForkShared));
  // of each slot: its holders but one, the requests whose open page it is, the first of these; and the
  // slots that nobody holds any more
  int32_t* const shares = kLocal ? local : p.shares_out;
  int32_t* const open = kLocal ? local + p.kv_slots : p.open;
  int32_t* const first = kLocal ? local + 2 * p.kv_slots : p.first;
  int32_t* const pushed = kLocal ? local + 3 * p.kv_slots : p.pushed;
  const int tid = threadIdx.x, part = Team::part(), n = p.n_req;
  const int lane = tid & 31, warp = part * kPartWarps + (tid >> 5);
  wait_before();
  const int cap = (int)min((int64_t)p.max_pages * kPageTokens, (int64_t)INT_MAX);
  bool bad = false;
  auto length = [&](int b) {
    const int v = p.len_in[b], c = min(max(v, 0), cap);
    bad |= v != c;
    return c;
  };
  const int n_free = min(max(*p.n_free_in, 0), p.free_cap);
  const Stretch mine(p.kv_slots, part, Team::parts);
  for (int i = mine.begin + tid; i < mine.end; i += kPartThreads) {
    if (kLocal || p.shares_in != p.shares_out) shares[i] = p.shares_in[i];
    open[i] = 0;
    first[i] = INT_MAX;
  }
  // ---- what each request asks for (every part for itself)
  for (int b = tid; b < n; b += kPartThreads) {
    const int own = length(b);
    int s = p.source[b], keep = 0, state = kNone;
    if (s == -1) {
      s = b;  // ends
    } else if (s < 0 || s >= n) {
      state = kRefused;
    } else {
      const int asked = p.len_keep ? p.len_keep[b] : INT_MAX, len = length(s);
      keep = p.len_keep ? asked : len;
      if (keep < 0 || keep > len) state = kRefused;
    }
    if (state == kRefused) {
      s = b;
      keep = own;
    } else if (s == b && keep == own) {
      state = kSame;
    }
    S.source[b] = s;
    S.keep[b] = keep;
    S.fresh[b] = state;
    S.page[b] = state == kNone && (keep & 63) ? p.table_in[(int64_t)s * p.max_pages + (keep >> 6)] : -1;
  }
  __syncthreads();
  Team::meet();

  // ---- holders: some warps to a request, or some requests to a warp
  const int warps = Team::parts * kPartWarps, team = max(1, warps / n);
  auto valid = [&](int x) {
    const bool ok = x >= 0 && x < p.kv_slots;
    bad |= !ok;
    return ok;
  };
  for (int b = warp / team; b < n && warp < warps / team * team; b += warps / team) {
    if (S.fresh[b] != kNone) continue;
    const int32_t* const own = p.table_in + (int64_t)b * p.max_pages;
    const int32_t* const from = p.table_in + (int64_t)S.source[b] * p.max_pages;
    const int lost = pages_of(length(b)), kept = S.keep[b] >> 6;
    for (int j = (warp % team) * 32 + lane; j < max(lost, kept); j += team * 32) {
      const int x = j < lost ? own[j] : -1, y = j < kept ? from[j] : -1;
      if (j < lost && j < kept && x == y) continue;
      if (j < lost && valid(x)) atomicSub(shares + x, 1);
      if (j < kept && valid(y)) atomicAdd(shares + y, 1);
    }
    if (warp % team == 0 && lane == 0 && (S.keep[b] & 63) && valid(S.page[b])) {
      atomicAdd(open + S.page[b], 1);
      atomicMin(first + S.page[b], b);
    }
  }
  Team::meet();

  // ---- slots: who keeps an open page, and which pages nobody holds
  auto freed = [&](int i) { return Team::get(shares + i) < 0 && Team::get(open + i) == 0; };
  int before, at, all;
  if (!kLocal) count_flags<kLocal>(mine, part, S.counts, p.counts, freed, before, at, all);
  if (kLocal) at = 0;
  // the highest is pushed first: those before are above
  for (int i0 = mine.end; i0 > mine.begin; i0 -= kPartThreads) {
    const int i = i0 - 1 - tid;
    const bool here = i >= mine.begin, gone = here && freed(i);
    int total;
    const int rank = rank_in_block(gone, S.counts, total);
    if (gone) pushed[at + rank] = i;
    at += total;
    if (!here) continue;
    const int base = Team::get(shares + i) + 1;
    bad |= base < 0;
    if (base <= 0) shares[i] = 0;
    else first[i] = -1;  // others hold it: nobody writes on
    if (kLocal) p.shares_out[i] = max(base - 1, 0);
  }
  if (kLocal) all = at;
  Team::meet();

  // ---- new slots for the pages that are copied, in request order (every part for itself)
  const int there = min(n_free + all, p.free_cap);
  int taken = 0;
  for (int b0 = 0; b0 < n; b0 += kPartThreads) {
    const int b = b0 + tid;
    bool asks = false, lost = false;
    int x = -1;
    if (b < n && S.fresh[b] == kNone && (S.keep[b] & 63)) {
      x = S.page[b];
      if (valid(x)) asks = Team::get(first + x) != b;
      else lost = true;
    }
    int total;
    const int rank = taken + rank_in_block(asks, S.counts, total);
    taken += total;
    // the stack's entries that this call pushed are not in free_slots yet
    const int from = there - 1 - rank;
    int got = kNone;
    if (asks && rank < there) {
      got = from < n_free ? p.free_slots[from] : Team::get(pushed + from - n_free);
      lost = !valid(got);  // an entry that is no slot: taken off the stack, and nobody's
    }
    lost |= asks && rank >= there;
    if (b >= n) continue;
    const bool copied = asks && !lost, refused = lost || S.fresh[b] == kRefused;
    if (lost) S.keep[b] &= ~63;
    if (S.fresh[b] == kNone || lost) S.fresh[b] = copied ? got : kNone;
    if (part == 0) {
      p.len_out[b] = S.keep[b];
      p.granted[b] = !refused;
      p.copy_src[b] = copied ? x : -1;
      p.copy_dst[b] = copied ? got : -1;
    }
  }
  const int left = there - min(taken, there);
  for (int i = n_free + part * kPartThreads + tid; i < left; i += Team::parts * kPartThreads)
    p.free_slots[i] = Team::get(pushed + i - n_free);
  if (part == 0 && tid == 0) {
    *p.n_free_out = left;
    bad |= n_free + all > p.free_cap;
  }
  __syncthreads();

  // ---- the new table rows
  for (int b = warp / team; b < n && warp < warps / team * team; b += warps / team) {
    const int32_t* const from = p.table_in + (int64_t)S.source[b] * p.max_pages;
    int32_t* const to = p.table_out + (int64_t)b * p.max_pages;
    const int pages = pages_of(S.keep[b]), fresh = S.fresh[b];
    for (int j = (warp % team) * 32 + lane; j < pages; j += team * 32)
      to[j] = fresh >= 0 && j == pages - 1 ? fresh : from[j];
  }
  if (bad) atomicOr(p.status, kStatusBadSlot);
}

// ------------------------------------------------------------- compaction
// The r-th lowest free slot takes the page of the r-th highest slot in use, while that is above it
// and r is below max_copies.  Then the stack holds the free slots, the lowest on top.
constexpr int kHeld = 0, kFree = 1, kTaken = 2;  // marks: in use, free, free and taken by a page

template <bool kLocal>
__global__ void __launch_bounds__(kPartThreads, 1) compact_kernel(const CompactParams p) {
  using Team = ::tpk::Team<kLocal>;
  extern __shared__ __align__(16) uint8_t raw[];
  int32_t* const local = reinterpret_cast<int32_t*>(raw);
  __shared__ int counts[kPartWarps];
  // of each slot: its mark, and where its page goes
  int32_t* const mark = kLocal ? local : p.mark;
  int32_t* const moved = kLocal ? local + p.kv_slots : p.new_slot;
  // the lists of the moves
  int32_t* const src = kLocal ? local + 2 * p.kv_slots : p.copy_src;
  int32_t* const dst = kLocal ? local + 3 * p.kv_slots : p.copy_dst;
  const int tid = threadIdx.x, lane = tid & 31, part = Team::part(), slots = p.kv_slots;
  const int step = Team::parts * kPartThreads, thread = part * kPartThreads + tid;
  wait_before();
  const int n_free = min(max(*p.n_free_in, 0), p.free_cap);
  const int most = min(p.max_copies, slots);  // entries of the lists that may be moves
  bool bad = false;
  for (int i = thread; i < slots; i += step) mark[i] = kHeld;
  for (int i = thread; i < most; i += step) src[i] = dst[i] = -1;
  for (int i = most + thread; i < p.max_copies; i += step) p.copy_src[i] = p.copy_dst[i] = -1;
  Team::meet();
  for (int i = thread; i < n_free; i += step) {
    const int x = p.free_in[i];
    if (x >= 0 && x < slots) mark[x] = kFree; else bad = true;
  }
  Team::meet();

  // ---- both lists: free slots from the bottom, slots in use from the top
  const Stretch mine(slots, part, Team::parts);
  int low, behind, all_free;  // free slots below this stretch, above it, in all
  count_flags<kLocal>(mine, part, counts, p.counts, [&](int i) { return Team::get(mark + i) == kFree; }, low, behind, all_free);
  const int held = slots - all_free;
  for (int i0 = mine.begin; i0 < mine.end; i0 += kPartThreads) {
    const int i = i0 + tid;
    const bool here = i < mine.end, is_free = here && Team::get(mark + i) == kFree;
    int total;
    const int below = low + rank_in_block(is_free, counts, total);
    low += total;
    if (!here) continue;
    moved[i] = is_free ? -1 : i;
    const int above = held - (i - below) - 1;  // slots in use above this one
    if (is_free && below < most) dst[below] = i;
    if (!is_free && above < most) src[above] = i;
  }
  Team::meet();

  // ---- the moves: those of the front of both lists
  auto goes = [&](int r) {
    const int s = Team::get(src + r), d = Team::get(dst + r);
    return d >= 0 && d < s;
  };
  if (thread == 0 && (most == 0 || !goes(0))) *p.n_copies = 0;
  for (int r = thread; r < most; r += step) {
    const bool go = goes(r);
    if (go) {
      const int s = Team::get(src + r), d = Team::get(dst + r);
      moved[s] = d;
      mark[d] = kTaken;
      // (an entry of the lists' rest is no move before and after it is cleared)
      if (r + 1 == most || !goes(r + 1)) *p.n_copies = r + 1;
    } else if (!kLocal) {
      src[r] = dst[r] = -1;
    }
    if (kLocal) {
      p.copy_src[r] = go ? src[r] : -1;
      p.copy_dst[r] = go ? dst[r] : -1;
    }
  }
  Team::meet();

  // ---- holders and the stack
  auto empty = [&](int i) {
    const int m = Team::get(mark + i);
    return m == kFree || (m == kHeld && Team::get(moved + i) != i);
  };
  int before, at, left;
  if (!kLocal) count_flags<kLocal>(mine, part, counts, p.counts + kParts, empty, before, at, left);
  if (kLocal) at = 0;
  for (int i0 = mine.end; i0 > mine.begin; i0 -= kPartThreads) {  // the highest at the bottom
    const int i = i0 - 1 - tid;
    const bool here = i >= mine.begin, is_empty = here && empty(i);
    int total;
    const int rank = rank_in_block(is_empty, counts, total);
    if (is_empty && at + rank < p.free_cap) p.free_out[at + rank] = i;
    at += total;
    if (!here) continue;
    const int m = Team::get(mark + i), to = Team::get(moved + i);
    // each slot in use brings its own holders along: no slot that is read here is written by another
    if (m == kHeld && to != i) p.shares_out[to] = p.shares_in[i];
    if (is_empty) p.shares_out[i] = 0;
    else if (m == kHeld && p.shares_in != p.shares_out) p.shares_out[i] = p.shares_in[i];
    if (kLocal) p.new_slot[i] = to;
  }
  if (kLocal) left = at;
  if (thread == 0) {
    *p.n_free_out = min(left, p.free_cap);
    bad |= left > p.free_cap;
  }

  // ---- the table rows
  const int cap = (int)min((int64_t)p.max_pages * kPageTokens, (int64_t)INT_MAX);
  const int warp = thread >> 5, warps = step / 32, team = max(1, warps / p.n_req);
  for (int b = warp / team; b < p.n_req && warp < warps / team * team; b += warps / team) {
    const int v = p.n_tokens[b], c = min(max(v, 0), cap);
    bad |= v != c;
    const int64_t row = (int64_t)b * p.max_pages;
    for (int j = (warp % team) * 32 + lane; j < pages_of(c); j += team * 32) {
      const int x = p.table_in[row + j], y = x >= 0 && x < slots ? Team::get(moved + x) : -1;
      bad |= y < 0;  // out of the pool, or on the stack: left as it is
      p.table_out[row + j] = y < 0 ? x : y;
    }
  }
  if (bad) atomicOr(p.status, kStatusBadSlot);
}

// ------------------------------------------------------------------ copies
// A block finds the pairs that are copies (kList entries at a time), then takes every gridDim-th
// piece of their pages in all pools: kCopyBytes together, each thread's loads in flight at once.
// Measured: 2,944 pages of 131 KB in four pools (3.1 GB) 491 us, 6.3 TB/s; 300 copies of 80 sources in
// 16 pools (629 MB written) 149 us.  (Four or sixteen loads a thread, two to eight blocks an SM, and
// loading a piece once for several copies of it in a row: within 4 %.)
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyBytes = kCopyThreads * kCopyUnroll * 16;
constexpr int kList = 2048;
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PagesCopyParams p) {
  __shared__ int2 list[kList];
  __shared__ int warp_counts[kCopyThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pieces = (int)((p.page_bytes + kCopyBytes - 1) / kCopyBytes);
  wait_before();
  int64_t turn = blockIdx.x;  // the block's next piece, counted from the current entries' first
  for (int e0 = 0; e0 < p.n_pages; e0 += kList) {
    const int n = min(kList, p.n_pages - e0);
    int found = 0;
    for (int i0 = 0; i0 < n; i0 += kCopyThreads) {
      const int i = i0 + tid;
      int s = -1, d = -1;
      if (i < n) {
        s = p.src[e0 + i];
        d = p.dst[e0 + i];
      }
      bool live = s >= 0 && d >= 0 && s != d;
      if (live && (s >= p.kv_slots || d >= p.kv_slots)) {
        live = false;
        if (blockIdx.x == 0) atomicOr(p.status, kStatusBadSlot);
      }
      const unsigned votes = __ballot_sync(0xffffffffu, live);
      __syncthreads();
      if (lane == 0) warp_counts[warp] = __popc(votes);
      __syncthreads();
      int before = found;
      for (int w = 0; w < kCopyThreads / 32; ++w) {
        if (w < warp) before += warp_counts[w];
        found += warp_counts[w];
      }
      if (live) list[before + __popc(votes & ((1u << lane) - 1))] = make_int2(s, d);
    }
    __syncthreads();
    const int64_t units = (int64_t)found * p.n_pools * pieces;
    for (; turn < units; turn += gridDim.x) {
      // neighbouring blocks take neighbouring pieces of a page
      const int piece = (int)(turn % pieces), rest = (int)(turn / pieces);
      const int2 pair = list[rest / p.n_pools];
      uint8_t* const pool = p.pools[rest % p.n_pools];
      const int64_t from = (int64_t)piece * kCopyBytes;
      const int words = (int)min((int64_t)kCopyBytes, p.page_bytes - from) / 16;
      const uint4* const src = reinterpret_cast<const uint4*>(pool + pair.x * p.page_bytes + from);
      uint4* const dst = reinterpret_cast<uint4*>(pool + pair.y * p.page_bytes + from);
      uint4 v[kCopyUnroll];
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u)
        if (u * kCopyThreads + tid < words) v[u] = src[u * kCopyThreads + tid];
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u)
        if (u * kCopyThreads + tid < words) dst[u * kCopyThreads + tid] = v[u];
    }
    turn -= units;
    __syncthreads();  // the list has been read
  }
}

// One block, or one cluster of kParts.
template <bool kLocal, typename P>
static cudaError_t launch_team(void (*kernel)(P), size_t smem, cudaStream_t stream, const P& p) {
  if (kLocal) return launch_early(kernel, 1, kPartThreads, smem, stream, p);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kParts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kParts);
  cfg.blockDim = dim3(kPartThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Shared memory of one block's arrays: four words for each slot.
static size_t local_bytes(int64_t slots) { return 4 * sizeof(int32_t) * slots; }
// Whether one block takes a call.  Its time grows with the slots, the requests (its 32 warps take one each)
// and the entries that rows hold, a cluster's hardly: 40 requests, or 14 in a compaction, cost it what 1,600
// and 560 slots do.  One block and the cluster, us, half of the requests forked:
//   requests x pages, slots      fork           compaction
//   64 x 56, 4,000               8.5   11.0     9.1   13.2
//   128 x 28, 4,000              9.6   11.0     9.8   13.4
//   256 x 1, 500                 10.2   9.6     8.5   12.0
//   64 x 112, 8,000              12.3  11.3     14.5  13.8
//   512 x 3, 2,000               17.9  12.0     14.8  13.5
//   4,000 x 2, 6,050             113   30.5     84    23.7
// What rows hold is not known here, and tables are mostly wider: their width counts only for what it may cost (64
// rows of the same 500 pages 17.8 and 11.2 us, of 1,000 31 and 12.8; 16 rows of 10 pages in a table as wide 4.9
// and 10.5).
constexpr int kForkRequest = 40, kForkMost = 9200, kCompactRequest = 14, kCompactMost = 8000;
static bool one_block(int n_req, int max_pages, int kv_slots, int request, int most) {
  return kv_slots <= kLocalSlots && (int64_t)n_req * max_pages <= kLocalEntries && kv_slots + request * n_req <= most;
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t e = once.run([] {
    const cudaError_t x = cudaFuncSetAttribute(fork_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(sizeof(ForkShared) + local_bytes(kLocalSlots)));
    return x != cudaSuccess ? x : cudaFuncSetAttribute(fork_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)sizeof(ForkShared));
  });
  if (e != cudaSuccess) return e;
  return one_block(p.n_req, p.max_pages, p.kv_slots, kForkRequest, kForkMost)
             ? launch_team<true>(fork_kernel<true>, sizeof(ForkShared) + local_bytes(p.kv_slots), stream, p)
             : launch_team<false>(fork_kernel<false>, sizeof(ForkShared), stream, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(compact_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)local_bytes(kLocalSlots));
  });
  if (e != cudaSuccess) return e;
  return one_block(p.n_req, p.max_pages, p.kv_slots, kCompactRequest, kCompactMost)
             ? launch_team<true>(compact_kernel<true>, local_bytes(p.kv_slots), stream, p)
             : launch_team<false>(compact_kernel<false>, 0, stream, p);
}

int device_sms();

cudaError_t launch_pages_copy(const PagesCopyParams& p, cudaStream_t stream) {
  // four blocks an SM keep 128 KB of loads in flight there
  const int64_t pieces = (p.page_bytes + kCopyBytes - 1) / kCopyBytes * p.n_pools * p.n_pages;
  const int blocks = (int)min(pieces, (int64_t)4 * device_sms());
  return launch_early(pages_copy_kernel, blocks, kCopyThreads, 0, stream, p);
}

}  // namespace tpk
