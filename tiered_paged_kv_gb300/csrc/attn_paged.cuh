// Attention of few query rows over paged keys and values whose lengths live on the
// device: one new token per request, or a handful of query tokens per request.
//
// A run is 8 or 16 query rows of one (request, KV head): the G heads of a new token, or
// (token, head) pairs of cross attention.  Every run of a request reads the same pages
// and costs that many units and kRunCost more (its queries and its join), so request b
// costs (pages_b + kRunCost) * runs_b; the units are numbered request by request, run by
// run, a run's own cost first.  Each of the N blocks of the launch takes an equal range
// of those numbers, whatever the lengths: the device stays evenly loaded and the split
// needs no host-side lengths.  A run inside one block's range is written out at once;
// one that crosses ranges leaves a partial (running maximum, sum, unnormalised o) in
// the block's two workspace slots -- slot 0: a run entered in the middle, slot 1: one
// left before its end -- and the fold kernel joins the partials in block order.  Where tables
// are short (split_whole) a block takes one run whole, and there is no fold.
//
// Within a block a producer warp walks the range and feeds a ring of page stages by TMA
// (64 tokens of keys and of values, 128-byte swizzle, a box per 16 tokens); four consumer
// warps take 16 of the 64 tokens each and keep their own online softmax, joined when a run
// ends.  Boxes outside the request's span are neither copied nor computed: 96 windows of
// 1000 tokens, 8 x 5 heads of 128, 66.9 -> 64.4 us.
// Both products run on mma.sync m16n8k16 with float32 accumulators (struct Rows).  The
// weights enter PV as two 16-bit planes (the rounded weight and what the rounding left:
// about 16 bits in bfloat16; 22 in float16, and at its lower end 2^-40 of the largest weight),
// so they add no error of their own next to the rounding of the output.  A tensor tile of 128 rows would hold 8 or 16 useful ones; the few rows make the
// kernel bound by HBM (4 H D bytes per attended token against 4 H G D operations).
//
// Through windows (kWindowed) a request's pages are its first ones and, behind a gap, those from its
// first query's window on; they are numbered, split and joined as if the gap were not there (120
// requests of up to 30,000 tokens, windows of 4,000 and 70 first tokens, 4 x 8 heads of 256: 101 us,
// 6.1 TB/s).  Over shared prefixes (kSharedPrefix) the requests that are numbered are the groups'
// prefixes, then what each request has of its own; a last kernel joins the two (cross_shared.cu; four
// answers to a prompt of 1,900 tokens, 8 x 4 heads of 128: 12.6 us).  Where row tiles take the prefixes, what
// requests have of their own is a launch like a decode's (kOwnTokens).
//
// Measured: 16 requests of 32,000 tokens at head sizes 64, 128, 256: 6.8, 6.9, 6.9 TB/s; one
// request of 131,072 tokens (4 x 8 heads of 256, 537 MB) 86 us, 6.2 TB/s; one of 200 tokens
// 7.4 us.
#pragma once
#include "paged.cuh"

namespace tpk {

constexpr float kEmpty = -__builtin_huge_valf();
constexpr int kConsumers = 4;
constexpr int kPagedThreads = (kConsumers + 1) * 32;

template <int D, bool kMany>  // kMany: a block per SM more, of a stage less
struct SplitCfg {
  static_assert(!kMany || D <= 128, "kMany");
  static constexpr int kPageBytes = kPageTokens * D * 2;   // keys or values of one page
  static constexpr int kStageBytes = 2 * kPageBytes;
  static constexpr int kBoxBytes = kBoxRows * D * 2;       // one warp's keys or values
  static constexpr int kStages = (D == 64 ? 4 : 3) - kMany;
  static constexpr int kBlocksPerSm = split_blocks(D) + kMany;
  static constexpr int kJoin = D == 256 ? 256 : D == 64 && kMany ? 32 : 64;  // channels joined at a time
  // floats a row, which spread the 8 rows (or the 4 lanes' row pairs) over the banks
  template <bool kSmall>
  static constexpr int kJoinStride = kJoin + (kSmall ? 4 : 8);
  static constexpr int kJoinBytes = kConsumers * 8 * kJoinStride<false> * 4;
  static constexpr int kSharedBytes = 768;  // SplitShared
  static constexpr int kSmem = kStages * kStageBytes + kJoinBytes + kSharedBytes;
  // shared memory of an SM, less what each block takes besides
  static_assert(kBlocksPerSm * (kSmem + 1024) <= 228 * 1024, "blocks per SM");
};

struct SplitShared {
  uint64_t full[4];
  uint64_t empty[4];
  int valid[4];
  float m[kConsumers][kRowTile];
  float l[kConsumers][kRowTile];
  int64_t scan[kPagedThreads / 32];
  int64_t base;  // more than kScanned requests: first unit of the one the block starts in
  int first;     // that request
};

// The pages that a request's queries see, in order: the first `sink_pages` of the table row (none
// unless windowed), then those from token `lo` on.
template <int kSpan>
struct Seen {
  int lo, hi;            // the span; tokens from hi on are not seen
  int sink_pages, skip;  // pages between the first ones and the span's
  // page i of them
  __device__ __forceinline__ int page(int i) const {
    return kSpan != kWindowed ? (lo >> 6) + i : i < sink_pages ? i : i + skip;
  }
};

constexpr int kRunCost = 3;

// Shared prefixes: a request of the numbering is a group's prefix, or what a request does not share.
struct VirtualReq {
  int lo, hi;                 // tokens [lo, hi) of the table row
  uint8_t first, count, row;  // whose queries these are, and that row
};
constexpr int kVirtual = 96;  // of them; query rows and table rows fit a byte

// The requests of a launch: their query rows, runs, pages and units.
template <int kSpan>
struct Batch {
  const PagedParams& p;
  const VirtualReq* v;  // shared prefixes only

  __device__ __forceinline__ void rows(int b, int& first, int& count) const {
    if (kSpan == kSharedPrefix) {
      first = v[b].first;
      count = v[b].count;
    } else {
      request_rows(p, b, first, count);
    }
  }
  __device__ __forceinline__ int runs(int b) const {
    int first, count;
    rows(b, first, count);
    return p.H * (int)(((int64_t)count * p.G + p.run_rows - 1) >> (p.run_rows == 8 ? 3 : 4));
  }
  __device__ __forceinline__ int pages(int b, Seen<kSpan>& s) const {
    if (kSpan == kSharedPrefix) {
      s.lo = v[b].lo;
      s.hi = v[b].hi;
    } else {
      request_span(p, b, s.lo, s.hi);
    }
    s.sink_pages = 0;
    if (kSpan == kWindowed) {  // from the first query token's window on
      int first, count;
      rows(b, first, count);
      s.lo = min(max(max(s.hi - count + 1, 0) - p.window, 0), s.hi);
      s.sink_pages = min((min(p.sinks, s.lo) + 63) >> 6, s.lo >> 6);
    }
    s.skip = (s.lo >> 6) - s.sink_pages;
    return s.hi > s.lo ? s.sink_pages + ((s.hi + 63) >> 6) - (s.lo >> 6) : 0;
  }
  __device__ __forceinline__ int64_t units(int b) const {
    Seen<kSpan> seen;
    const int n = pages(b, seen);
    return n > 0 ? (int64_t)(n + kRunCost) * runs(b) : 0;
  }
  __device__ __forceinline__ const int32_t* table(int b) const {
    return p.table + (int64_t)(kSpan == kSharedPrefix ? v[b].row : b) * p.max_pages;
  }
  // where the results of its first query token go: behind a launch over shared prefixes those of the
  // prefixes come first, then those of what is not shared
  __device__ __forceinline__ int out(int b, int first) const {
    return kSpan == kSharedPrefix && b >= p.n_grp ? first + p.n_q : first;
  }
};

__device__ __forceinline__ int64_t per_block(int64_t total, int blocks) {
  const int64_t per = (total + blocks - 1) / blocks;
  return per < kRunCost + 1 ? kRunCost + 1 : per;
}

// The numbering of up to kScanned requests by one warp: lane i has requests 4 i .. 4 i + 3.
struct Numbers {
  int64_t total, before;  // all units; those before this lane's requests
  int64_t units[4];
  template <typename F>
  __device__ __forceinline__ void load(const PagedParams& p, F of_request) {
    const int lane = threadIdx.x & 31;
    int64_t mine = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      units[x] = 4 * lane + x < p.n_req ? of_request(p, 4 * lane + x) : 0;
      mine += units[x];
    }
    int64_t inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += up;
    }
    before = inc - mine;
    total = __shfl_sync(0xffffffffu, inc, 31);
  }
  // The request that holds unit `at` (below total) and the units before it.
  __device__ __forceinline__ void find(int64_t at, int& b, int64_t& base) const {
    int64_t begin = before, here = -1;
    int mine = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (at >= begin && at < begin + units[x]) {
        here = begin;
        mine = 4 * (threadIdx.x & 31) + x;
      }
      begin += units[x];
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here >= 0)) - 1;
    b = __shfl_sync(0xffffffffu, mine, src);
    base = __shfl_sync(0xffffffffu, here, src);
  }
};

// One stretch of pages of one run.
template <int kSpan>
struct Segment {
  int b, run, page, count, pages;  // pages [page, page + count) of the run's `pages`
  Seen<kSpan> seen;
};

// Steps through a block's range, segment by segment.
template <int kSpan>
struct Walk {
  int64_t at, end, base;
  int b;
  __device__ __forceinline__ bool next(const Batch<kSpan>& batch, Segment<kSpan>& s) {
    while (at < end) {
      s.pages = batch.pages(b, s.seen);
      const int units = s.pages + kRunCost;
      const int64_t work = s.pages > 0 ? (int64_t)units * batch.runs(b) : 0;
      if (at >= base + work) {
        base += work;
        ++b;
        continue;
      }
      const int64_t local = at - base;
      s.b = b;
      s.run = (int)(local / units);
      const int from = (int)(local - (int64_t)s.run * units);
      const int to = (int)min((int64_t)units, end - at + from);
      at += to - from;
      s.page = max(from - kRunCost, 0);
      s.count = to - kRunCost - s.page;
      if (s.count > 0) return true;  // else the range ends within the run's own cost
    }
    return false;
  }
};

template <typename T>
__device__ __forceinline__ void store_pair(const PagedParams& p, int64_t row, int head, int D, int c, float x, float y) {
  const int64_t at = row * p.o_stride + (int64_t)head * D + c;
  if (p.o_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.o) + at) = make_float2(x, y);
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at) = T::pack(x, y);
}

// A row's log-sum, or its maximum and sum.
template <int kSpan>
__device__ __forceinline__ void store_sum(const PagedParams& p, int64_t row, float M, float L) {
  if (leaves_sums(kSpan)) reinterpret_cast<float2*>(p.lse)[row] = make_float2(M, L);
  else p.lse[row] = L == 0.f ? kEmpty : (M + log2f(L)) * kLn2;
}
// What a row's values are multiplied by.
template <int kSpan>
__device__ __forceinline__ float over_sum(float L) { return leaves_sums(kSpan) ? 1.f : L == 0.f ? 0.f : 1.f / L; }

// Row r of a run: its query token and query head; false past the run's last row.
__device__ __forceinline__ bool run_row(const PagedParams& p, int first, int count, int h, int tile, int r, int& token,
                                        int& head) {
  // 32 bits do: a call has at most 2^31 query rows
  const uint32_t i = (uint32_t)tile * p.run_rows + r;
  if (i >= (uint32_t)count * (uint32_t)p.G) return false;
  const uint32_t t = i / (uint32_t)p.G;
  token = first + (int)t;
  head = h * p.G + (int)(i - t * (uint32_t)p.G);
  return true;
}

// One warp's share of a run, as 32 lanes (g, t) = (lane / 4, lane % 4) hold it: every lane has
// two of the run's rows, row(0) and row(1), and of those some tokens' scores and some
// channels' output.
// Up to 8 rows are the narrow side of m16n8k16: S^T = K Q^T (16 tokens x 8 rows; rows 2t and
// 2t + 1), O^T += V^T P^T (16 channels x 8 rows), P^T being S^T transposed in registers.  A
// third fewer steps than 8 rows of 16, and half the accumulators: 400 requests of 200 to 300
// tokens, 8 heads of 256: 171 us (207 as the wide side); one of 200 tokens 7.6 (9.0).
// Up to 16 rows are the wide side: S = Q K^T, O += P V, rows g and g + 8; as two narrow tiles
// 96 requests of 1000 tokens, 8 heads of 128, take 77 us instead of 73.
template <typename T, int D, bool kSmall, int kSpan>
struct Rows {
  static constexpr int kAcc = kSmall ? D / 16 : D / 8;
  uint32_t q[D / 16][kSmall ? 2 : 4];
  int see_lo[2], see_hi[2];  // the tokens each row sees (besides the first ones, windowed)
  float acc[kAcc][4];
  float m[2], l[2];  // l: of this lane's tokens
  int g, t, r8, i8;  // r8, i8: row r8 of matrix i8 in ldmatrix

  __device__ __forceinline__ explicit Rows(int lane) : g(lane >> 2), t(lane & 3), r8(lane & 7), i8(lane >> 3) {}
  __device__ __forceinline__ int row(int e) const { return kSmall ? 2 * t + e : g + 8 * e; }
  // Joins x over the lanes that share this lane's rows.
  template <typename F>
  __device__ __forceinline__ static float over_lanes(float x, F f) {
#pragma unroll
    for (int d = kSmall ? 4 : 1; d < (kSmall ? 32 : 4); d <<= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
  }

  __device__ __forceinline__ void start(const PagedParams& p, int first, int count, int h, int tile, const Seen<kSpan>& seen) {
    const int tok_lo = seen.lo, tok_hi = seen.hi;
    int token, head;
#pragma unroll
    for (int e = 0; e < (kSmall ? 1 : 2); ++e) {
      const bool live = run_row(p, first, count, h, tile, g + 8 * e, token, head);
      const uint32_t* src =
          reinterpret_cast<const uint32_t*>(p.q + (live ? (int64_t)token * p.q_stride + (int64_t)head * D : 0));
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][e] = live ? src[8 * k + t] : 0;
        q[k][e + (kSmall ? 1 : 2)] = live ? src[8 * k + t + 4] : 0;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool live = run_row(p, first, count, h, tile, row(e), token, head);
      see_lo[e] = tok_lo;
      see_hi[e] = live ? tok_hi : tok_lo;
      if (live && p.range) {
        see_lo[e] = max(tok_lo, p.range[2 * (int64_t)token]);
        see_hi[e] = min(tok_hi, p.range[2 * (int64_t)token + 1]);
      }
      if (kSpan == kSharedPrefix && live) see_hi[e] = min(tok_hi, max(p.own_lens[token], 0));
      if (kSpan == kWindowed) {  // the query token's position is its place among the request's last ones
        see_hi[e] = live ? max(tok_hi - count + (token - first) + 1, 0) : 0;
        see_lo[e] = max(see_hi[e] - p.window, 0);
      }
      m[e] = kEmpty;
      l[e] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < kAcc; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
  }

  // Folds in 16 tokens from tok0 on, whose keys and values start at ks and vs: of each 64
  // channels kBoxRows rows of 128 bytes.
  __device__ __forceinline__ void tokens(const PagedParams& p, uint32_t ks, uint32_t vs, int tok0) {
    // ---- scores, two chains of matrix steps a tile
    constexpr int kTiles = kSmall ? 1 : 2;  // of 8 tokens, in the wide form
    float sc[kTiles][2][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][x][e] = 0.f;
    const int k_half = kSmall ? i8 & 1 : i8 >> 1, k_piece = kSmall ? i8 >> 1 : i8 & 1;
    const uint32_t krow = ks + (k_half * 8 + r8) * 128;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t kf[4];
      const int c = 2 * k + k_piece;  // 16-byte piece of the row
      ldmatrix_x4(kf, krow + (c >> 3) * (kBoxRows * 128) + (((c & 7) ^ r8) << 4));
      if constexpr (kSmall) {
        T::mma(sc[0][k & 1], kf, q[k][0], q[k][1]);
      } else {
        T::mma(sc[0][k & 1], q[k], kf[0], kf[1]);
        T::mma(sc[1][k & 1], q[k], kf[2], kf[3]);
      }
    }
    // ---- online softmax in base 2, each row for itself
    constexpr int kMine = kSmall ? 2 : 4;  // tokens of a row in this lane
    float x[2][kMine];
    bool grows = false;  // beyond the maximum so far
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int y = 0; y < kMine; ++y) {
        const int tok = tok0 + (kSmall ? g + 8 * y : 8 * (y >> 1) + 2 * t + (y & 1));
        const int n = kSmall ? 0 : y >> 1, at = kSmall ? 2 * y + e : 2 * e + (y & 1);
        const bool seen = (tok >= see_lo[e] || (kSpan == kWindowed && tok < p.sinks)) && tok < see_hi[e];
        x[e][y] = seen ? __fmul_rn(sc[n][0][at] + sc[n][1][at], p.qscale) : kEmpty;
        grows = grows || x[e][y] > m[e];
      }
    // Three steps over 8 lanes wait for the vote, two over 4 do not.
    const bool scaled = __any_sync(0xffffffffu, grows);
    float scale[2];
    if (!kSmall || scaled) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = m[e];
#pragma unroll
        for (int y = 0; y < kMine; ++y) top = fmaxf(top, x[e][y]);
        top = over_lanes(top, [](float a, float b) { return fmaxf(a, b); });
        scale[e] = m[e] == kEmpty ? 0.f : exp2f(m[e] - top);
        m[e] = top;
        l[e] *= scale[e];
      }
    }
    if (scaled) {
#pragma unroll
      for (int c = 0; c < kAcc; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][e] *= scale[kSmall ? e & 1 : e >> 1];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float ref = m[e] == kEmpty ? 0.f : m[e];
      float sum = 0.f;
#pragma unroll
      for (int y = 0; y < kMine; ++y) {
        x[e][y] = exp2f(x[e][y] - ref);
        sum += x[e][y];
      }
      l[e] += sum;
    }
    // ---- o += weights * values, in two planes: the rounded weights, and what that left
    constexpr float kScale = 1 << T::kWeightBits;  // put takes it out again
    uint32_t hi[4], lw[4];
#pragma unroll
    for (int i = 0; i < (kSmall ? 2 : 4); ++i) {
      float a, b;
      if constexpr (kSmall) {
        a = x[0][i];
        b = x[1][i];
      } else {
        a = x[i & 1][i & 2];
        b = x[i & 1][(i & 2) + 1];
      }
      a *= kScale;
      b *= kScale;
      hi[i] = T::pack(a, b);
      const float2 back = T::unpack(hi[i]);
      lw[i] = T::pack(a - back.x, b - back.y);
      if constexpr (kSmall) {
        hi[i] = transpose8(hi[i]);
        lw[i] = transpose8(lw[i]);
      }
    }
    const int v_half = kSmall ? i8 >> 1 : i8 & 1, v_piece = kSmall ? i8 & 1 : i8 >> 1;
    const uint32_t vrow = vs + (v_half * 8 + r8) * 128;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t vf[4];
      const int c = 2 * n + v_piece;
      ldmatrix_x4_trans(vf, vrow + (c >> 3) * (kBoxRows * 128) + (((c & 7) ^ r8) << 4));
      if constexpr (kSmall) {
        T::mma(acc[n], vf, hi[0], hi[1]);
        T::mma(acc[n], vf, lw[0], lw[1]);
      } else {
        T::mma(acc[2 * n], hi, vf[0], vf[1]);
        T::mma(acc[2 * n + 1], hi, vf[2], vf[3]);
        T::mma(acc[2 * n], lw, vf[0], vf[1]);
        T::mma(acc[2 * n + 1], lw, vf[2], vf[3]);
      }
    }
  }

  // Puts kJoin channels from c0 on, times f, into `to` (8 rows of `stride` floats): the run's
  // rows 8 pass .. 8 pass + 7.
  template <int kJoin>
  __device__ __forceinline__ void put(float* to, int stride, int c0, int pass, const float (&f)[2]) const {
    if constexpr (kSmall) {
#pragma unroll
      for (int c = 0; c < kJoin / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          to[(2 * t + (e & 1)) * stride + 16 * c + 8 * (e >> 1) + g] = acc[c0 / 16 + c][e] * f[e & 1];
    } else {
#pragma unroll
      for (int c = 0; c < kJoin / 8; ++c)
        *reinterpret_cast<float2*>(to + g * stride + 8 * c + 2 * t) =
            make_float2(acc[c0 / 8 + c][2 * pass] * f[pass], acc[c0 / 8 + c][2 * pass + 1] * f[pass]);
    }
  }
};

// The numbering's requests of a launch over shared prefixes: the p.n_grp groups (p.q_off their first
// requests, p.lens their prefixes), then what each of the p.n_q requests has of its own.  A prefix
// is read from the row of the first request that has the most of it.  For the whole block.
__device__ __forceinline__ void shared_requests(const PagedParams& p, VirtualReq* v) {
  const int cap = p.max_pages * 64;
  bool bad = false;
  auto tokens = [&](int b) {
    const int n = p.own_lens[b], c = min(max(n, 0), cap);
    bad |= n != c;
    return c;
  };
  for (int g = threadIdx.x; g < p.n_grp; g += kPagedThreads) {
    int first, count, most = 0, row = 0;
    request_rows(p, g, first, count);
    const int shared = p.lens[g], n = min(max(shared, 0), cap);
    bad |= shared != n;
    if (count < 2) count = 0;  // nobody to share with
    for (int i = 0; i < count; ++i) {
      const int own = min(tokens(first + i), n);
      if (own > most) {
        most = own;
        row = first + i;
      }
    }
    v[g] = {0, most, (uint8_t)first, (uint8_t)count, (uint8_t)row};
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.n_q; b += kPagedThreads) {
    int begin = 0;
    for (int g = 0; g < p.n_grp; ++g)
      if (b >= v[g].first && b < v[g].first + v[g].count) begin = v[g].hi;
    v[p.n_grp + b] = {begin, tokens(b), (uint8_t)b, 1, (uint8_t)b};
    if (blockIdx.x == 0) p.own_begin[b] = begin;
  }
  if (bad) atomicOr(p.status, kStatusBadSlot);
  __syncthreads();
}

// The second bound asks for the registers of kBlocksPerSm blocks.  In the wide form at
// D = 128 two fit without it (167 registers); with it the compiler spills (96 requests of
// 1000 tokens, 16 rows: 73 us without, 80 with; asking for one block, which takes 214, 91).
template <typename T, int D, bool kSmall, bool kMany, int kSpan>
__global__ void __launch_bounds__(kPagedThreads, D == 128 && !kSmall ? 0 : split_blocks(D) + kMany)
    split_kernel(const __grid_constant__ PagedParams p) {
  using C = SplitCfg<D, kMany>;
  extern __shared__ __align__(1024) uint8_t stages[];
  float* join = reinterpret_cast<float*>(stages + C::kStages * C::kStageBytes);
  static_assert(sizeof(SplitShared) <= C::kSharedBytes, "SplitShared");
  SplitShared& S = *reinterpret_cast<SplitShared*>(stages + C::kStages * C::kStageBytes + C::kJoinBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_u32(stages) & 1023) {  // the swizzle counts on it
    wait_before();
    if (tid == 0) {
      atomicOr(p.status, kStatusTimeout);
      if (kSpan == kSharedPrefix || !p.whole) p.cuts[blockIdx.x].parts = 0;
    }
    return;
  }

  // ---- the numbering: this block's range
  if (tid == kConsumers * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.vmap) : "memory");
  }
  if (tid < C::kStages) {
    mbar_init(&S.full[tid], 1);
    mbar_init(&S.empty[tid], kConsumers);
    fence_mbar_init();
  }
  wait_before();
  VirtualReq* const virtuals = reinterpret_cast<VirtualReq*>(stages + C::kStages * C::kStageBytes + C::kJoinBytes + C::kSharedBytes);
  if (kSpan == kSharedPrefix) shared_requests(p, virtuals);
  const Batch<kSpan> batch{p, virtuals};
  Walk<kSpan> walk;
  int64_t per = 0;  // numbers of a range
  if (kSpan != kSharedPrefix && p.whole) {
    // a block per run: nothing to join, and nothing to number if every request has as many
    int64_t run;
    if (p.q_off) {
      Numbers numbers;
      numbers.load(p, [&](const PagedParams&, int b) { return batch.runs(b); });
      if (blockIdx.x >= numbers.total) return;  // the grid is an upper bound
      numbers.find(blockIdx.x, walk.b, run);
      run = blockIdx.x - run;
    } else {
      const int runs = batch.runs(0);
      walk.b = blockIdx.x / runs;
      run = blockIdx.x - walk.b * runs;
    }
    __syncthreads();
    int first, count;
    Seen<kSpan> seen;
    const int runs = batch.runs(walk.b);
    const int pages = batch.pages(walk.b, seen);
    walk.base = 0;
    walk.at = run * (pages + kRunCost);
    walk.end = walk.at + pages + kRunCost;
    if (pages == 0) {
      batch.rows(walk.b, first, count);
      const int tiles = runs / p.H, h = (int)run / tiles;
      for (int i = tid; i < p.run_rows * (D / 2); i += kPagedThreads) {
        int token, head;
        if (!run_row(p, batch.out(walk.b, first), count, h, (int)run - h * tiles, i / (D / 2), token, head)) continue;
        store_pair<T>(p, token, head, D, i % (D / 2) * 2, 0.f, 0.f);
        if (i % (D / 2) == 0) store_sum<kSpan>(p, (int64_t)token * p.H * p.G + head, kEmpty, 0.f);
      }
      return;
    }
  } else {
    start_next();
    int64_t lo, hi;
    if (p.n_req <= kScanned) {
      Numbers numbers;
      numbers.load(p, [&](const PagedParams&, int b) { return batch.units(b); });
      per = per_block(numbers.total, gridDim.x);
      lo = min(per * blockIdx.x, numbers.total);
      hi = min(lo + per, numbers.total);
      if (lo < hi) numbers.find(lo, walk.b, walk.base);
      __syncthreads();
    } else {
      const int each = (p.n_req + kPagedThreads - 1) / kPagedThreads;
      const int b0 = min(tid * each, p.n_req), b1 = min(b0 + each, p.n_req);
      int64_t mine = 0;
      for (int b = b0; b < b1; ++b) mine += batch.units(b);
      int64_t inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += up;
      }
      if (lane == 31) S.scan[warp] = inc;
      __syncthreads();
      int64_t total = 0, before = inc - mine;
#pragma unroll
      for (int w = 0; w < kPagedThreads / 32; ++w) {
        if (w < warp) before += S.scan[w];
        total += S.scan[w];
      }
      per = per_block(total, gridDim.x);
      lo = min(per * blockIdx.x, total);
      hi = min(lo + per, total);
      if (lo < hi && lo >= before && lo < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
          const int64_t work = batch.units(b);
          if (lo >= at && lo < at + work) {
            S.first = b;
            S.base = at;
          }
          at += work;
        }
      }
      __syncthreads();
      walk.b = S.first;
      walk.base = S.base;
    }
    walk.at = lo;
    walk.end = hi;
    if (tid == 0) p.cuts[blockIdx.x].parts = 0;  // until this block leaves a run before its end

  // ---- requests that attend nothing
  for (int b = blockIdx.x; b < p.n_req; b += gridDim.x) {
    int first, count;
    Seen<kSpan> seen;
    if (batch.pages(b, seen) > 0) continue;
    batch.rows(b, first, count);
    first = batch.out(b, first);
    const int HQ = p.H * p.G;
    for (int64_t i = tid; i < (int64_t)count * HQ * (D / 2); i += kPagedThreads) {
      const int64_t r = i / (D / 2);
      store_pair<T>(p, first + r / HQ, (int)(r % HQ), D, (int)(i % (D / 2)) * 2, 0.f, 0.f);
    }
    for (int64_t i = tid; i < (int64_t)count * HQ; i += kPagedThreads) store_sum<kSpan>(p, (int64_t)first * HQ + i, kEmpty, 0.f);
  }
    if (lo >= hi) return;
  }

  Segment<kSpan> s;
  if (warp == kConsumers) {
    // ------------------------------------------------------------- producer
    const bool stalled = (int)blockIdx.x == p.stall_unit;
    int item = 0;
    bool dead = false;
    while (!dead && walk.next(batch, s)) {
      const int tiles = batch.runs(s.b) / p.H;
      const int h = s.run / tiles;
      const int32_t* row = batch.table(s.b);
      for (int j0 = 0; j0 < s.count && !dead; j0 += 32) {
        const int entry = j0 + lane < s.count ? row[s.seen.page(s.page + j0 + lane)] : 0;
        const int n = min(32, s.count - j0);
        for (int j = 0; j < n; ++j, ++item) {
          const int tok0 = s.seen.page(s.page + j0 + j) * kPageTokens;  // the page's first token
          const int64_t slot = __shfl_sync(0xffffffffu, entry, j);
          const int st = item % C::kStages;
          if (item >= C::kStages) {
            const bool ok = mbar_wait(&S.empty[st], ((item / C::kStages) - 1) & 1, p.status, p.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) {
              dead = true;
              break;
            }
          }
          if (elect_one() && !(item == 0 && stalled)) {
            const bool ok = slot >= 0 && slot < p.kv_slots;
            S.valid[st] = ok;
            if (ok) {
              uint8_t* k = stages + st * C::kStageBytes;
              const int y = (int)((slot * p.H + h) * kPageTokens);
              // the boxes with tokens of the span (and those between the first tokens and the span,
              // if both are in this page)
              int x0 = max(s.seen.lo - tok0, 0) / kBoxRows;
              int x1 = (min(s.seen.hi - tok0, kPageTokens) + kBoxRows - 1) / kBoxRows;
              if (kSpan == kWindowed && tok0 < p.sinks) {
                x0 = 0;
                if (tok0 + kPageTokens <= s.seen.lo) x1 = (min(p.sinks - tok0, kPageTokens) + kBoxRows - 1) / kBoxRows;
              }
              mbar_arrive_expect_tx(&S.full[st], (x1 - x0) * 2 * C::kBoxBytes);
              for (int x = x0; x < x1; ++x) tma_load_3d(k + x * C::kBoxBytes, &p.kmap, 0, y + x * kBoxRows, 0, &S.full[st]);
              for (int x = x0; x < x1; ++x)
                tma_load_3d(k + C::kPageBytes + x * C::kBoxBytes, &p.vmap, 0, y + x * kBoxRows, 0, &S.full[st]);
            } else {
              atomicOr(p.status, kStatusBadSlot);
              mbar_arrive(&S.full[st]);
            }
          }
          __syncwarp();
        }
      }
    }
    // No copy is in flight when the block ends, whoever gave up: the latest item of each stage has
    // landed (those before it had, or its stage would not have been free).
    for (int i = max(stalled ? 1 : 0, item - C::kStages); i < item; ++i)
      mbar_wait(&S.full[i % C::kStages], (i / C::kStages) & 1, p.status, p.wait_ns);
    return;
  }

  // --------------------------------------------------------------- consumers
  Rows<T, D, kSmall, kSpan> rows(lane);
  bool dead = false;
  int item = 0;  // pages of this block so far
  while (walk.next(batch, s)) {
    const int tok_lo = s.seen.lo, tok_hi = s.seen.hi;
    // tokens that no row sees: their rows in the pages may hold anything
    auto hidden = [&](int t) { return (t < tok_lo && !(kSpan == kWindowed && t < p.sinks)) || t >= tok_hi; };
    int first, count;
    batch.rows(s.b, first, count);
    const int out = batch.out(s.b, first);  // its rows in the output
    const int tiles = batch.runs(s.b) / p.H;
    const int h = s.run / tiles, tile = s.run - h * tiles;
    rows.start(p, first, count, h, tile, s.seen);

    for (int j = 0; j < s.count; ++j, ++item) {
      const int st = item % C::kStages;
      if (!dead) {
        const bool ok = mbar_wait(&S.full[st], (item / C::kStages) & 1, p.status, p.wait_ns);
        dead = !__all_sync(0xffffffffu, ok);
      }
      const int tok0 = s.seen.page(s.page + j) * kPageTokens + warp * 16;  // this warp's first token
      const bool some = tok0 + 16 > tok_lo || (kSpan == kWindowed && tok0 < p.sinks);
      if (!dead && S.valid[st] && tok0 < tok_hi && some) {
        uint8_t* ks = stages + st * C::kStageBytes + warp * C::kBoxBytes;
        uint8_t* vs = ks + C::kPageBytes;
        // rows outside the request's span may hold NaN: their weight is 0, their
        // values are cleared
        if ((tok0 < tok_lo && !(kSpan == kWindowed && tok0 + 16 <= p.sinks)) || tok0 + 16 > tok_hi) {
          for (int x = lane; x < 16 * (D / 8); x += 32) {
            const int r = x / (D / 8), c = x % (D / 8);
            if (hidden(tok0 + r))
              *reinterpret_cast<uint4*>(vs + (c >> 3) * (kBoxRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();  // the stage is filled by TMA again later
          __syncwarp();
        }
        rows.tokens(p, smem_u32(ks), smem_u32(vs), tok0);
      }
      __syncwarp();
      // a stage that was not seen full is not free: the producer then stops too
      if (lane == 0 && !dead) mbar_arrive(&S.empty[st]);
    }

    // ---- join the warps' states, 8 rows at a time by kPer threads each
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float l = rows.over_lanes(rows.l[e], [](float a, float b) { return a + b; });
      if ((kSmall ? rows.g : rows.t) == 0) {
        S.m[warp][rows.row(e)] = rows.m[e];
        S.l[warp][rows.row(e)] = l;
      }
    }
    named_barrier(1, kConsumers * 32);
    const bool whole = s.count == s.pages;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (s.page == 0 ? 1 : 0);
    const int HQ = p.H * p.G;
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = kEmpty;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, S.m[w][rows.row(e)]);
      f[e] = (rows.m[e] == kEmpty ? 0.f : exp2f(rows.m[e] - top)) * (1.f / (1 << T::kWeightBits));
    }
    constexpr int kPer = kConsumers * 4, kStride = C::template kJoinStride<kSmall>;
#pragma unroll
    for (int pass = 0; pass < (kSmall ? 1 : 2); ++pass) {
      const int row = tid / kPer, r = row + 8 * pass;
      // A maximum skips NaN, a sum does not: a row whose scores are NaN has no maximum, yet a sum
      // that is not 0, which tells it from a row that sees nothing.
      float M = kEmpty, L = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, S.m[w][r]);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) L += exp2f(S.m[w][r] - (M == kEmpty ? 0.f : M)) * S.l[w][r];
      int token, head;
      const bool write = run_row(p, out, count, h, tile, r, token, head) && !dead;
      const float inv = whole ? over_sum<kSpan>(L) : 1.f;
      // the join's record: this block has the run's first page and not its last
      if (tid == 0 && pass == 0 && !whole && s.page == 0)
        p.cuts[blockIdx.x] = {out, count, h, tile, (int)((s.pages - s.count - 1) / per) + 2};
      if (write && tid % kPer == 0) {
        if (whole) {
          store_sum<kSpan>(p, (int64_t)token * HQ + head, M, L);
        } else {
          p.part_ml[slot * kRowTile + r] = M;
          p.part_ml[(2 * (int64_t)gridDim.x + slot) * kRowTile + r] = L;
        }
      }
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += C::kJoin) {
        rows.template put<C::kJoin>(join + warp * 8 * kStride, kStride, c0, pass, f);
        named_barrier(1, kConsumers * 32);
        if (write) {
#pragma unroll
          for (int c = (tid % kPer) * 4; c < C::kJoin; c += kPer * 4) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) {
              const float4 v = *reinterpret_cast<const float4*>(join + (w * 8 + row) * kStride + c);
              o.x += v.x;
              o.y += v.y;
              o.z += v.z;
              o.w += v.w;
            }
            if (whole) {
              store_pair<T>(p, token, head, D, c0 + c, o.x * inv, o.y * inv);
              store_pair<T>(p, token, head, D, c0 + c + 2, o.z * inv, o.w * inv);
            } else {
              *reinterpret_cast<float4*>(p.part_o + (slot * kRowTile + r) * D + c0 + c) = o;
            }
          }
        }
        named_barrier(1, kConsumers * 32);
      }
    }
  }
}

// Joins the partials of the runs that cross block ranges: block (i, r) takes row r of the
// run that range i begins and leaves, if there is one (its record).  It reads nothing before
// its wait: only there are the writes of the launches before it sure to be seen.  The
// partials' maxima are read at once, one a thread; then every thread sums its four
// channels over the partials in block order, eight loads in flight.
constexpr int kFoldParts = 64;  // weights held at a time
template <typename T, int D, int kSpan>
__global__ void __launch_bounds__(64) fold_paged_kernel(const __grid_constant__ PagedParams p, int blocks, int rows) {
  __shared__ float weight[kFoldParts];
  __shared__ float red[2];
  const int i = blockIdx.x / rows, r = blockIdx.x % rows, tid = threadIdx.x;
  // block i left the run before its end, the others entered it in the middle
  auto slot = [&](int k) { return (2 * (int64_t)(i + k) + (k == 0 ? 1 : 0)) * kRowTile + r; };
  const float* part_l = p.part_ml + 2 * (int64_t)blocks * kRowTile;
  wait_before();
  const RunCut cut = p.cuts[i];
  const int n = cut.parts;  // blocks i .. i + n - 1 hold a piece
  int token, head;
  if (n == 0 || !run_row(p, cut.first, cut.count, cut.h, cut.tile, r, token, head)) return;
  float M = kEmpty;
  for (int k = tid; k < n; k += 64) M = fmaxf(M, p.part_ml[slot(k)]);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  if ((tid & 31) == 0) red[tid >> 5] = M;
  __syncthreads();
  M = fmaxf(red[0], red[1]);
  const float ref = M == kEmpty ? 0.f : M;
  float L = 0.f;
  constexpr int kVec = D >= 256 ? 4 : D / 64;  // channels of a thread
  float o[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) o[e] = 0.f;
  const int c = tid * kVec;
  for (int k0 = 0; k0 < n; k0 += kFoldParts) {
    const int cnt = min(kFoldParts, n - k0);
    __syncthreads();
    if (tid < cnt) weight[tid] = exp2f(p.part_ml[slot(k0 + tid)] - ref);
    float mine = tid < cnt ? weight[tid] * part_l[slot(k0 + tid)] : 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = mine;
    __syncthreads();
    L += red[0] + red[1];
    for (int j0 = 0; j0 < cnt; j0 += 8) {
      float v[8][kVec];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < cnt) {
          const float* src = p.part_o + slot(k0 + j0 + j) * D + c;
          if constexpr (kVec == 4) *reinterpret_cast<float4*>(v[j]) = *reinterpret_cast<const float4*>(src);
          else if constexpr (kVec == 2) *reinterpret_cast<float2*>(v[j]) = *reinterpret_cast<const float2*>(src);
          else v[j][0] = *src;
        }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < cnt) {
          const float w = weight[j0 + j];
#pragma unroll
          for (int e = 0; e < kVec; ++e) o[e] += w * v[j][e];
        }
    }
  }
  const float inv = over_sum<kSpan>(L);
  if constexpr (kVec == 1) {
    const float x = o[0] * inv, y = __shfl_down_sync(0xffffffffu, x, 1);
    if ((tid & 1) == 0) store_pair<T>(p, token, head, D, c, x, y);
  } else {
#pragma unroll
    for (int e = 0; e < kVec; e += 2) store_pair<T>(p, token, head, D, c + e, o[e] * inv, o[e + 1] * inv);
  }
  if (tid == 0) store_sum<kSpan>(p, (int64_t)token * p.H * p.G + head, M, L);
}

int device_sms();

// Runs of a launch: a decode's, an upper bound of cross attention's.
inline int64_t most_runs(const PagedParams& p) {
  const int64_t each = (p.G + p.run_rows - 1) / p.run_rows;
  return p.H * (p.q_off ? (int64_t)p.n_q * p.G / p.run_rows + p.n_req : p.n_req * each);
}

template <typename T, int D, bool kSmall, bool kMany, int kSpan>
cudaError_t launch_split(const PagedParams& p, cudaStream_t stream) {
  using C = SplitCfg<D, kMany>;
  constexpr int extra = kSpan == kSharedPrefix ? kVirtual * (int)sizeof(VirtualReq) : 0;
  static_assert(C::kBlocksPerSm * (C::kSmem + extra + 1024) <= 228 * 1024, "blocks per SM");
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(split_kernel<T, D, kSmall, kMany, kSpan>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem + extra);
  });
  if (e != cudaSuccess) return e;
  const int blocks = p.whole ? (int)most_runs(p) : min(device_sms() * C::kBlocksPerSm, kPagedMaxBlocks);
  e = launch_early(split_kernel<T, D, kSmall, kMany, kSpan>, blocks, kPagedThreads, C::kSmem + extra, stream, p);
  if (e != cudaSuccess || p.whole || blocks == 1) return e;
  // the fold's blocks may start while the last ranges still run: they wait for them
  const int rows = p.q_off ? p.run_rows : min(p.G, p.run_rows);
  return launch_early(fold_paged_kernel<T, D, kSpan>, (blocks - 1) * rows, 64, 0, stream, p, blocks, rows);
}

template <typename T, int D, int kSpan>
cudaError_t launch_rows(const PagedParams& p, cudaStream_t stream) {
  if constexpr (D <= 128 && kSpan != kSharedPrefix) {
    // A block per SM more, of a stage less, for whole runs: 40 requests of 1500 tokens, 8 heads of
    // 128, one wave instead of two, 51 -> 41 us; 64 of 1500, heads of 64, 44 -> 34; 400 of 250, 128,
    // 84 -> 75; not where its waves leave more of the device idle (64 of 1500, 128: 62 and 74),
    // nor where runs are cut (96 of 5000, 128: 290 and 296).
    constexpr int kFew = split_blocks(D);
    auto waves = [&](int64_t blocks) { return (most_runs(p) + blocks * kTileBlocks - 1) / (blocks * kTileBlocks); };
    if (p.run_rows == 8 && p.whole && waves(kFew) > 1 && 10 * (kFew + 1) * waves(kFew + 1) <= 11 * kFew * waves(kFew))
      return launch_split<T, D, true, true, kSpan>(p, stream);
  }
  return p.run_rows == 8 ? launch_split<T, D, true, false, kSpan>(p, stream) : launch_split<T, D, false, false, kSpan>(p, stream);
}

template <typename T, int kSpan>
cudaError_t launch_dim(const PagedParams& p, int D, cudaStream_t stream) {
  return D == 64 ? launch_rows<T, 64, kSpan>(p, stream) : D == 128 ? launch_rows<T, 128, kSpan>(p, stream)
                                                            : launch_rows<T, 256, kSpan>(p, stream);
}

// span_pages: pages that a request's queries see, at most.
template <int kSpan>
cudaError_t launch_by_rows(PagedParams& p, int span_pages, int D, int dtype, cudaStream_t stream) {
  auto whole = [&] { return split_whole(p.q_off, p.n_req, p.q_off ? (int64_t)p.n_req * p.H : most_runs(p), span_pages); };
  // Runs of 8 rows where requests have no more; also where few of them are cut (read_twice),
  // and where none is and all are resident at once, a page's second reader finding it in L2
  // (one request of 500 tokens, 8 x 16 heads of 256: 10.4 us, 16.0 with runs of 16; nine: 11.0
  // and 16.3; where not all are resident, 18 of 300: 17.3 with runs of 8, 13.8 with 16).
  p.run_rows = 8;
  if ((int64_t)p.n_q * p.G > 8 * (int64_t)p.n_req &&
      !(whole() ? most_runs(p) <= split_blocks(D) * kTileBlocks : read_twice(most_runs(p), span_pages, D)))
    p.run_rows = kRowTile;
  p.whole = whole();
  return dtype == 0 ? launch_dim<Bf16, kSpan>(p, D, stream) : launch_dim<F16, kSpan>(p, D, stream);
}

}  // namespace tpk
