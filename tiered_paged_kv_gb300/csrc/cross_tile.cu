// Cross attention of many query rows on the fifth-generation tensor cores.
//
// An item is one or two 128-row tiles of one (request, KV head), rows being packed (query
// token, head) pairs: two tiles share the keys and values for D <= 128, unless the
// requests have fewer rows; TMEM holds one for D = 256.  The keys and values pass once,
// 128 tokens (two pages) at a time, through a ring of shared-memory slots filled by TMA.
// Per key tile S = Q K^T goes to TMEM, two threads per row turn 64 scores each into
// weights (online softmax in base 2), write them over S in the input type, and O += P V
// runs with P read from TMEM as the A operand.
//
// Roles: a loader warp finds the items (the block's own, then blocks not started that it
// takes over from the launch queue, longest requests first), describes them to the
// others and loads keys and values (at D = 256 a warp of its own loads the values); one
// warp loads queries; one thread issues the matrix instructions; 8 or 16 warps do the
// softmax and write the rows.  All of them run ahead into the next item as far as their
// buffers let them, so that its start hides behind the end of the one before.
//
// The tensor core is kept busy while a softmax runs by a second score buffer: of the
// other row tile with two, of the next keys with one.  The issuing thread runs
// QK(0), QK(1), then PV(i), QK(i + 2), ...  The matrix instructions of one thread execute
// in order, so QK(i + 2) may overwrite the buffer that PV(i) reads its weights from.
// PV(i) starts on half of each row's weights while the other half is being formed.
//
// The reference of a row's weights moves only when its maximum has grown by more than 2^8
// (2^4 in float16), so the pass that rescales O in TMEM is rare.  In float16 it stands 2^11
// below the maximum it was taken from: weights stay below 2^15, and those far below the
// maximum are held to 2^-36 of it (struct F16).  Weights are rounded once to the input type -- as the
// tensor core needs them beside V -- while their sum is kept unrounded in float32: the
// rounding of a weight is of the size of the output's own.
//
// Few query rows leave the device empty, so the keys can be split into `splits` parts
// per item; parts leave (maximum, sum, O) in the workspace and a fold joins them in part
// order.  Bound: the tensor cores (4 D operations per score); for D = 64 the exponentials, for
// D = 256 the arrival of keys and values (128 rows use 128 KB in 2,048 matrix cycles).
//
// Measured: two requests of 4,096 tokens, 8,192 states, 8 x 4 heads: 922, 1,546 and 1,332
// TFLOP/s at D = 64, 128, 256; eight requests of 300 to 1,500 tokens, 1,601 to 6,404
// states at D = 128 311 us, 1,340 TFLOP/s.
#include "paged.cuh"

namespace tpk {

constexpr float kNone = -__builtin_huge_valf();
// log2 of a row's largest weight over its reference, and of how much more it may become
template <typename T>
constexpr int kLift = T::kWeightBits > 0 ? T::kWeightBits - 4 : 0;
template <typename T>
constexpr int kSlack = T::kWeightBits > 0 ? 4 : 8;
// References from here on are refused: the maximum is rounded when it is scaled, the scores are not
// (a fused step forms scaled score - reference), so a weight may be 2^(half a float32 step) over the
// largest meant.  At 2^23 that is 2^0.5 and float16 still holds it, at 2^29 2^32 (bfloat16); further
// out weights pass the type's range or all vanish.  Such a row becomes NaN, o and lse.  (Scaling and
// rounding the scores first where references are large cost the prompts 2-3 % wherever it was put.)
template <typename T>
__device__ __forceinline__ bool far_off(float m) {
  return fabsf(m) >= (T::kWeightBits > 0 ? 0x1p23f : 0x1p29f) && m != kNone;
}
constexpr int kKeys = 128;     // tokens of a key tile
constexpr uint32_t kTmemCols = 512;

template <int D, int kT>
struct TileCfg {
  static constexpr int kTiles = kT;
  static constexpr int kRows = kTiles * kTileRows;
  static constexpr int kSlotChannels = D < 128 ? D : 128;
  static constexpr int kSlotBytes = kKeys * kSlotChannels * 2;
  static constexpr int kParts = D / kSlotChannels;  // slots per key (or value) tile
  static constexpr int kSlots = D == 64 ? 8 : D == 128 && kT == 1 ? 6 : 5;
  static constexpr int kQBytes = kTileRows * D * 2;  // one tile
  static constexpr int kSharedBytes = 3 * 1024;      // TileShared
  static constexpr int kSmem = kSharedBytes + kTiles * kQBytes + kSlots * kSlotBytes;
  static constexpr int kSoftWarps = kTiles * 8;  // softmax: two threads per row
  static constexpr int kMma = kSoftWarps, kLoad = kMma + 1, kQuery = kLoad + 1;
  // At D = 256 one loader issues more slowly than the tensor core takes the tiles, and the
  // values get a warp of their own (72 -> 70 us at the clips); at 128 it costs 2 %.
  static constexpr bool kTwoLoaders = kParts == 2;
  static constexpr int kValues = kQuery + 1;
  static constexpr int kThreads = (kQuery + 1 + kTwoLoaders) * 32;
};

// One tile group of one (request, KV head), or one part of its keys.
struct Item {
  int id;       // its block number; -1: no more
  int first;    // its first query token
  int tokens;   // and how many of them it has: `per_tile` fill a row tile
  int h, len, b;
  int page0, page_end, nk;  // key tiles [0, nk) begin at page page0
  int last;     // 16-token groups of the last key tile that hold any token
};

struct TileShared {
  uint4 next;                      // the work taken over from a block not started
  uint64_t full[8], empty[8];      // ring of key and value slots
  uint64_t s_full[2];              // scores written (by score buffer)
  uint64_t p_half[2], p_full[2];   // weights of half of each row's pieces written, of all
  uint64_t pv_done, o_full[2], o_empty[2];  // a product ended (one tile), the last one; o read (by tile)
  uint64_t q_full, q_empty, tail, drain, taken;
  uint64_t item_full[2], item_empty[2];
  Item item[2];
  uint32_t tmem;
  // what the block must see land before it ends: by slot, the copies that complete its `full`; those
  // that complete `tail` and `q_full`
  int laps[8], tails, loads;
  int fine[2][8][2];               // [item parity][pair of warps][half]: waits met so far
  float half[4 * kTileRows];       // what the two threads of a row tell each other
};

// ------------------------------------------------------------ tcgen05 wrappers
__device__ __forceinline__ void tmem_alloc(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(kTmemCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(kTmemCols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D += A B with both operands in shared memory, or A in TMEM.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// 32 columns of this warp's 32 rows (lane = row) <-> 32 registers a thread.
__device__ __forceinline__ void tc_ld32(float* r, uint32_t addr) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const float* r) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
// After a wait: what follows may not be moved above it by the compiler, which does not
// know that a load's registers are filled only then.
template <int N>
__device__ __forceinline__ void tc_loaded(float (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}
// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 bytes, aligned to 32.
__device__ __forceinline__ void store32(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory operand descriptor, 128-byte swizzle: 8-row groups of 1024 bytes follow
// each other; 64-channel chunks are `leading` apart (read only where the channels are not
// the reduced dimension).  A later 16-byte piece is the descriptor plus one.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading) {
  const uint32_t lo = (addr & 0x3ffff) >> 4 | (leading >> 4) << 16;
  return (uint64_t)((1024 >> 4) | 1u << 14 | 2u << 29) << 32 | lo;
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Instruction descriptor: float32 accumulator, both inputs of one type, M = 128.
__device__ __forceinline__ constexpr uint32_t instruction(bool bf16, bool b_rows_reduced, int n) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_rows_reduced ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(kTileRows >> 4) << 24;
}

template <typename T>
struct IsBf16 {
  static constexpr bool value = false;
};
template <>
struct IsBf16<Bf16> {
  static constexpr bool value = true;
};

// Takes over a block that has not started: its number arrives at S.next and completes the
// barrier; or the news that none is left.
__device__ __forceinline__ void take_block(uint4* dst, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(dst)),
      "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ int taken_block(const uint4* src) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(src))
      : "memory");
  return got ? (int)x : -1;
}

struct Keys {
  static constexpr bool value = false;
};
struct Values {
  static constexpr bool value = true;
};
// Page-table entries of 16 key tiles, one a lane.
struct TableWindow {
  int32_t entry = -1;
  int window = -1;
};

// Finds the request of a tile group.  Lane i of the warp holds requests base + i and
// base + 32 + i: their query rows, lengths, groups, and the groups before them.
struct Requests {
  int per_group;           // query tokens of a group
  int base = -64, begin = 0, end = 0;  // groups [begin, end) are those of the 64 held
  int first[2], count[2], len[2], groups[2], before[2];

  __device__ __forceinline__ void load(const PagedParams& p, int lane) {
    int sum = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int b = base + 32 * x + lane;
      int lo;
      first[x] = count[x] = len[x] = 0;
      if (b < p.n_req) {
        request_rows(p, b, first[x], count[x]);
        request_span(p, b, lo, len[x]);
      }
      groups[x] = (count[x] + per_group - 1) / per_group;
      int inc = groups[x];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += up;
      }
      before[x] = begin + sum + inc - groups[x];
      sum += __shfl_sync(0xffffffffu, inc, 31);
    }
    end = begin + sum;
  }
  // Longest first: blocks start in index order, so the last ones to run are short.  (With
  // more than 64 requests their lengths even out.)
  __device__ __forceinline__ void sort(const PagedParams& p, int lane) {
    int b2[2] = {0, 0};
    for (int y = 0; y < p.n_req; ++y) {
      const int n = __shfl_sync(0xffffffffu, y < 32 ? len[0] : len[1], y & 31);
      const int g = __shfl_sync(0xffffffffu, y < 32 ? groups[0] : groups[1], y & 31);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (n > len[x] || (n == len[x] && y < 32 * x + lane)) b2[x] += g;
    }
    before[0] = b2[0];
    before[1] = b2[1];
  }
  // Fills in the request of group `want`; false past the last one.
  __device__ __forceinline__ bool find(const PagedParams& p, int lane, bool sorted, int want, Item& it) {
    if (base < 0 || want < begin) {
      base = begin = 0;
      load(p, lane);
      if (sorted) sort(p, lane);
    }
    while (want >= end) {
      if (base + 64 >= p.n_req) return false;
      base += 64;
      begin = end;
      load(p, lane);
    }
    const uint32_t m0 = __ballot_sync(0xffffffffu, want >= before[0] && want < before[0] + groups[0]);
    const uint32_t m1 = __ballot_sync(0xffffffffu, want >= before[1] && want < before[1] + groups[1]);
    const int src = (m0 ? __ffs(m0) : __ffs(m1)) - 1;
    const bool second = m0 == 0;
    it.b = base + (second ? 32 : 0) + src;
    const int t = (want - __shfl_sync(0xffffffffu, second ? before[1] : before[0], src)) * per_group;
    it.first = __shfl_sync(0xffffffffu, second ? first[1] : first[0], src) + t;
    it.tokens = min(__shfl_sync(0xffffffffu, second ? count[1] : count[0], src) - t, per_group);
    it.len = __shfl_sync(0xffffffffu, second ? len[1] : len[0], src);
    return true;
  }
};

template <typename T, int D, int kT>
__global__ void __launch_bounds__(TileCfg<D, kT>::kThreads, 1)
    tile_kernel(const __grid_constant__ PagedParams p, int splits) {
  using C = TileCfg<D, kT>;
  extern __shared__ __align__(1024) uint8_t raw[];
  static_assert(sizeof(TileShared) <= C::kSharedBytes, "TileShared");
  TileShared& S = *reinterpret_cast<TileShared*>(raw);
  uint8_t* qs = raw + C::kSharedBytes;
  uint8_t* slots = qs + C::kTiles * C::kQBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_u32(raw) & 1023) {  // the swizzle counts on it
    wait_before();
    if (tid == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  if (tid == 0) {
    S.tails = S.loads = 0;
#pragma unroll
    for (int i = 0; i < C::kSlots; ++i) {
      S.laps[i] = 0;
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_half[i], 256);
      mbar_init(&S.p_full[i], 256);
      mbar_init(&S.o_full[i], 1);
      mbar_init(&S.o_empty[i], 256);
      mbar_init(&S.item_full[i], 1);
      mbar_init(&S.item_empty[i], C::kSoftWarps + 2 + C::kTwoLoaders);
    }
    mbar_init(&S.pv_done, 1);
    mbar_init(&S.q_full, 1);
    mbar_init(&S.q_empty, 1);
    mbar_init(&S.tail, 1);
    mbar_init(&S.drain, 1);
    mbar_init(&S.taken, 1);
    fence_mbar_init();
  }
  if (tid == C::kLoad * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.vmap) : "memory");
  }
  wait_before();
  start_next();
  if (warp == C::kMma) tmem_alloc(&S.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int G = p.G, per_tile = kTileRows / G;  // query tokens of a row tile (rows past them are not used)
  // the next item for a whole warp; false if it did not come in time
  auto next_item = [&](int k, Item& it) {
    const bool ok =
        __all_sync(0xffffffffu, mbar_wait(&S.item_full[k & 1], k >> 1 & 1, p.status, p.wait_ns)) != 0;
    if (ok) it = S.item[k & 1];
    __syncwarp();
    if (ok && lane == 0) mbar_arrive(&S.item_empty[k & 1]);
    return ok;
  };

  // One key (or value) tile, two pages, into the kParts ring slots from position `pos` on (a
  // position is a slot and a lap)
  auto load_tile = [&](auto kind, const Item& it, TableWindow& w, int j, int pos, int& tails, bool& ok) {
    constexpr bool values = decltype(kind)::value;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, p.status, p.wait_ns)) != 0;
    };
    if (j >> 4 > w.window) {
      w.window = j >> 4;
      const int pg = it.page0 + 32 * w.window + lane;
      w.entry = pg < it.page_end ? p.table[(int64_t)it.b * p.max_pages + pg] : -1;
    }
    const int slot0 = __shfl_sync(0xffffffffu, w.entry, 2 * j & 31);
    const int slot1 = __shfl_sync(0xffffffffu, w.entry, (2 * j & 31) + 1);
    const unsigned n_slots = (unsigned)p.kv_slots;
    const bool there0 = (unsigned)slot0 < n_slots, there1 = (unsigned)slot1 < n_slots;
    const int n = there0 + there1;
    const bool second = it.page0 + 2 * j + 1 < it.page_end;  // the tile has a second page
    const int tok0 = (it.page0 + 2 * j) * kPageTokens;
    const bool bad = !there0 || (!there1 && second);
    if (bad && lane == 0) atomicOr(p.status, kStatusBadSlot);
    // values whose weight is 0 must not be NaN: rows past the last token in its 16-token
    // group (later groups are not multiplied), and pages not there
    const bool clear = values && (bad || (it.len - tok0 < kKeys && (it.len & 15)));
    const int y0 = (slot0 * p.H + it.h) * kPageTokens, y1 = (slot1 * p.H + it.h) * kPageTokens;
    const CUtensorMap* map = values ? &p.vmap : &p.kmap;
#pragma unroll
    for (int c = 0; c < C::kParts; ++c) {
      const int st = (pos + c) % C::kSlots, lap = (pos + c) / C::kSlots;
      if (lap > 0) wait(&S.empty[st], lap - 1);
      if (!ok) return;
      uint8_t* dst = slots + st * C::kSlotBytes;
      uint64_t* bar = clear ? &S.tail : &S.full[st];
      if (elect_one() && !(!values && pos == 0 && (int)blockIdx.x == p.stall_unit)) {
        if (clear) S.tails = tails + 1; else S.laps[st] = lap + 1;
        if (n > 0) mbar_arrive_expect_tx(bar, n * (C::kSlotBytes / 2));
        else mbar_arrive(bar);
#pragma unroll
        for (int ch = 0; ch < C::kSlotChannels; ch += 64) {
          uint8_t* to = dst + ch / 64 * (kKeys * 128);
          if (there0) tma_load_2d(to, map, c * C::kSlotChannels + ch, y0, bar);
          if (there1) tma_load_2d(to + kPageTokens * 128, map, c * C::kSlotChannels + ch, y1, bar);
        }
      }
      __syncwarp();
      if (clear) {
        wait(&S.tail, tails++);
        constexpr int kPieces = C::kSlotChannels / 8;
        const int piece = lane % kPieces;
        const int end = min(kKeys, max(0, it.len - tok0));  // rows that hold tokens
        const int last = bad ? kKeys : (end + 15) & ~15;
        for (int r = bad ? lane / kPieces : end + lane / kPieces; r < last; r += 32 / kPieces)
          if (r >= end || !(r < kPageTokens ? there0 : there1))
            *reinterpret_cast<uint4*>(dst + (piece >> 3) * (kKeys * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4)) =
                make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && ok) {
          S.laps[st] = lap + 1;
          mbar_arrive(&S.full[st]);
        }
      }
    }
  };
  // ring positions of key and value tile j of an item whose first position is `base`, in
  // the order the tensor core takes them
  auto k_pos = [&](const Item& it, int base, int j) {
    return base + C::kParts * (C::kTiles == 2 ? 2 * j : j == 0 ? 0 : 2 * j - 1);
  };
  auto v_pos = [&](const Item& it, int base, int j) {
    return base + C::kParts * (C::kTiles == 2 || j + 1 == it.nk ? 2 * j + 1 : 2 * j + 2);
  };

  if (warp == C::kMma) {
    // ------------------------------------------------------------ matrix issue
    // One elected lane runs all of it: nothing to keep the warp together for.  The key
    // and value tiles lie in the ring in the order they are taken here:
    // K0 V0 K1 V1 ... with two row tiles, K0 K1 V0 K2 V1 ... with one.
    if (elect_one()) {
      constexpr bool bf16 = IsBf16<T>::value;
      constexpr uint32_t id_qk = instruction(bf16, false, kKeys);
      constexpr uint32_t id_pv = instruction(bf16, true, C::kSlotChannels);
      const uint32_t empty = smem_u32(S.empty), s_full = smem_u32(S.s_full), o_full = smem_u32(S.o_full);
      const uint32_t q_empty = smem_u32(&S.q_empty), pv_done = smem_u32(&S.pv_done);
      const uint64_t q_op = operand(smem_u32(qs), 16);
      const uint64_t k_op = operand(smem_u32(slots), 16), v_op = operand(smem_u32(slots), kKeys * 128);
      constexpr uint64_t kSlotStep = C::kSlotBytes >> 4;
      int next = 0, phase = 0;        // ring position of the next tile
      int items = 0;                  // with work, so far
      int used[2] = {0, 0};           // items of each row tile so far
      int step[2] = {0, 0};           // steps of each score buffer so far
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) { ok = ok && mbar_wait(bar, parity & 1, p.status, p.wait_ns); };
      // the first slot of the next tile, once it has landed
      auto take = [&] {
        const int at = next;
#pragma unroll
        for (int c = 0; c < C::kParts; ++c) {
          wait(&S.full[next], phase);
          if (++next == C::kSlots) {
            next = 0;
            phase ^= 1;
          }
        }
        return at;
      };
      auto nth = [&](int at, int c) { return at + c < C::kSlots ? at + c : at + c - C::kSlots; };
      // scores of row tile x with the keys at `at`, into score buffer `buf`
      auto qk = [&](int x, int buf, int at, bool last) {
        const uint64_t q = q_op + x * (C::kQBytes >> 4);
#pragma unroll
        for (int c = 0; c < C::kParts; ++c) {
          const uint64_t k = k_op + nth(at, c) * kSlotStep;
#pragma unroll
          for (int i = 0; i < C::kSlotChannels / 16; ++i)  // 64-channel chunks of 16 KB, 32 bytes a step
            tc_mma_ss(tmem + buf * kKeys, q + (c * (C::kSlotChannels / 64) + i / 4) * (kTileRows * 8) + i % 4 * 2,
                      k + i / 4 * (kKeys * 8) + i % 4 * 2, id_qk, c > 0 || i > 0);
          if (last) tc_commit(empty + 8 * nth(at, c));
        }
        tc_commit(s_full + 8 * buf);
      };
      // o of row tile x += weights in buffer `buf` times the values at `at`: the first
      // halves of the rows' pieces as soon as they are there; `last`: no other row tile
      // needs the values; `groups`: 16-token groups that hold any token
      auto pv = [&](int x, int buf, int at, bool more, bool last, int groups) {
        if (!more) {  // o of the item before has been read
          if (used[x] > 0) wait(&S.o_empty[x], used[x] - 1);
          ++used[x];
        }
        const int n = step[buf]++;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          wait(s == 0 ? &S.p_half[buf] : &S.p_full[buf], n);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::kParts; ++c) {
            const uint64_t v = v_op + nth(at, c) * kSlotStep;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int i = (y >> 1) * 4 + 2 * s + (y & 1);  // 16 tokens: two 8-row groups
              if (i < groups)
                tc_mma_ts(tmem + 256 + x * 128 + c * 128, tmem + buf * kKeys + i / 4 * (kKeys / 2) + i % 4 * 8,
                          v + i * 128, id_pv, more || s > 0 || y > 0);
            }
            if (last && s == 1) tc_commit(empty + 8 * nth(at, c));
          }
        }
      };
      for (int k = 0; ok; ++k) {
        wait(&S.item_full[k & 1], k >> 1);
        if (!ok) break;
        const int id = S.item[k & 1].id, nk = S.item[k & 1].nk, tail = S.item[k & 1].last;
        const bool two = C::kTiles == 2 && S.item[k & 1].tokens > per_tile;
        mbar_arrive(&S.item_empty[k & 1]);
        if (id < 0) break;
        if (nk == 0) continue;
        wait(&S.q_full, items++);
        tc_fence_after();
        int ka = take();
        if (!ok) break;
        if (C::kTiles == 2) {
          qk(0, 0, ka, !two);
          if (two) qk(1, 1, ka, true);
          if (nk == 1) tc_commit(q_empty);
          for (int j = 0; j < nk && ok; ++j) {
            const int va = take();
            const bool more = j + 1 < nk;
            if (more) ka = take();
            if (!ok) break;
            pv(0, 0, va, j > 0, !two, more ? 8 : tail);
            if (!ok) break;
            if (more) qk(0, 0, ka, !two); else tc_commit(o_full);
            if (two) {
              pv(1, 1, va, j > 0, true, more ? 8 : tail);
              if (!ok) break;
              if (more) qk(1, 1, ka, true); else tc_commit(o_full + 8);
            }
            if (j + 2 == nk) tc_commit(q_empty);
          }
        } else {
          const int b0 = (step[0] + step[1]) & 1;  // score buffer of the first step
          qk(0, b0, ka, true);
          if (nk > 1) {
            ka = take();
            if (!ok) break;
            qk(0, b0 ^ 1, ka, true);
          }
          if (nk <= 2) tc_commit(q_empty);
          for (int j = 0; j < nk && ok; ++j) {
            const int va = take();
            const bool more = j + 2 < nk;
            if (more) ka = take();
            if (!ok) break;
            pv(0, b0 ^ (j & 1), va, j > 0, true, j + 1 < nk ? 8 : tail);
            if (!ok) break;
            tc_commit(pv_done);
            if (j + 1 == nk) tc_commit(o_full);
            if (more) {
              qk(0, b0 ^ (j & 1), ka, true);
              if (j + 3 == nk) tc_commit(q_empty);
            }
          }
        }
      }
      tc_commit(smem_u32(&S.drain));
      mbar_wait(&S.drain, 0, p.status, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == C::kLoad) {
    // -------------------------------------------------------- items, and their keys
    const bool sorted = splits == 1 && p.n_req <= 64;
    Requests requests;
    requests.per_group = C::kTiles * per_tile;
    int base = 0, tails = 0;  // ring positions before this item
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, p.status, p.wait_ns)) != 0;
    };
    int id = blockIdx.x;
    int asked = 0;
    for (int k = 0; ok; ++asked) {
      // Asked for near the end of an item's loads: asked earlier, a block would commit
      // itself to an item that another is free for first.
      bool open = true;
      auto ask = [&] {
        if (lane == 0) {
          mbar_arrive_expect_tx(&S.taken, 16);
          take_block(&S.next, &S.taken);
        }
        open = false;
      };
      // ---- what the item is
      Item it;
      const int part = id % splits;
      it.id = id;
      it.first = 0;
      it.h = id / splits % p.H;
      const bool found = requests.find(p, lane, sorted, id / splits / p.H, it);
      // the join's record, by the block of the group's first part
      if (splits > 1 && part == 0 && lane == 0) p.cuts[id / splits] = {it.first, found ? it.tokens : 0, it.h, 0, splits};
      if (found) {
        int clo = 0, chi = it.len;
        if (p.range) {  // what any of its rows sees
          clo = 0x7fffffff;
          chi = 0;
          for (int t = it.first + lane; t < it.first + it.tokens; t += 32) {
            const int a = max(0, p.range[2 * (int64_t)t]), e = min(it.len, p.range[2 * (int64_t)t + 1]);
            if (e > a) {
              clo = min(clo, a);
              chi = max(chi, e);
            }
          }
          clo = __reduce_min_sync(0xffffffffu, clo);
          chi = __reduce_max_sync(0xffffffffu, chi);
        }
        it.page0 = chi > clo ? clo >> 6 : 0;
        it.page_end = (chi + 63) >> 6;
        const int nk = chi > clo ? (it.page_end - it.page0 + 1) >> 1 : 0;
        const int k0 = (int)((unsigned)nk * (unsigned)part / (unsigned)splits);  // splits <= kTileBlocks, nk < 2^24
        const int k1 = (int)((unsigned)nk * (unsigned)(part + 1) / (unsigned)splits);
        it.page0 += 2 * k0;
        it.nk = k1 - k0;
        it.last = min(8, (min(it.len, it.page_end * kPageTokens) - (it.page0 + 2 * (it.nk - 1)) * kPageTokens + 15) >> 4);
        if (k >= 2) wait(&S.item_empty[k & 1], (k >> 1) - 1);
        if (ok && lane == 0) {
          S.item[k & 1] = it;
          mbar_arrive(&S.item_full[k & 1]);
        }
        __syncwarp();
        ++k;
        TableWindow w, w2;  // with one row tile the keys are one tile ahead
        for (int j = 0; j < it.nk && ok; ++j) {
          if (j + 4 == it.nk) ask();
          if (C::kTwoLoaders) {
            load_tile(Keys{}, it, w, j, k_pos(it, base, j), tails, ok);
            continue;
          }
          if (C::kTiles == 2 || j == 0) load_tile(Keys{}, it, w, j, k_pos(it, base, j), tails, ok);
          if (C::kTiles == 1 && j + 1 < it.nk && ok) load_tile(Keys{}, it, w2, j + 1, k_pos(it, base, j + 1), tails, ok);
          if (ok) load_tile(Values{}, it, w, j, v_pos(it, base, j), tails, ok);
        }
        base += 2 * C::kParts * it.nk;
      }
      if (open) ask();
      wait(&S.taken, asked);
      if (!ok) break;
      id = taken_block(&S.next);
      fence_async_smem();  // read before the next answer is written
      __syncwarp();
      if (id < 0) {
        if (k >= 2) wait(&S.item_empty[k & 1], (k >> 1) - 1);
        if (ok && lane == 0) {
          S.item[k & 1].id = -1;
          mbar_arrive(&S.item_full[k & 1]);
        }
        break;
      }
    }
    if (!ok) mbar_wait(&S.taken, asked & 1, p.status, p.wait_ns);
    __syncwarp();
  } else if (C::kTwoLoaders && warp == C::kValues) {
    // ------------------------------------------------------------------ values
    int base = 0, tails = 0;
    bool ok = true;
    Item it;
    for (int k = 0; ok && next_item(k, it) && it.id >= 0; ++k) {
      TableWindow w;
      for (int j = 0; j < it.nk && ok; ++j) load_tile(Values{}, it, w, j, v_pos(it, base, j), tails, ok);
      base += 2 * C::kParts * it.nk;
    }
    __syncwarp();
  } else if (warp == C::kQuery) {
    // ----------------------------------------------------------------- queries
    int items = 0;
    Item it;
    for (int k = 0; next_item(k, it) && it.id >= 0; ++k) {
      if (it.nk == 0) continue;
      if (items > 0 &&
          !__all_sync(0xffffffffu, mbar_wait(&S.q_empty, (items - 1) & 1, p.status, p.wait_ns)))
        break;
      ++items;
      // rows (token, head) of each tile; tokens past the request's are someone else's or,
      // past the last, zero: no row of theirs is written
      const int tiles = it.tokens > per_tile ? 2 : 1;
      if (elect_one()) {
        S.loads = items;
        mbar_arrive_expect_tx(&S.q_full, tiles * per_tile * G * D * 2);
        for (int x = 0; x < tiles; ++x)
#pragma unroll
          for (int c = 0; c < D; c += 64)
            tma_load_3d(qs + x * C::kQBytes + c / 64 * (kTileRows * 128), &p.qmap, c, it.h * G,
                        it.first + x * per_tile, &S.q_full);
      }
      __syncwarp();
    }
  } else {
    // ----------------------------------------------------------------- softmax
    // Warp w has rows 32 (w mod 4) .. of tile w / 8 (a warp reaches the TMEM rows of its
    // number mod 4 only) and keys 64 (w / 4 mod 2) .. of each key tile.
    const int tile = warp >> 3, half = warp >> 2 & 1, row = (warp & 3) * 32 + lane, hrow = tile * kTileRows + row;
    const float qscale = fabsf(p.qscale);  // its sign goes to the scores
    constexpr int kMine = kKeys / 2;       // keys of this thread's half
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's TMEM rows
    const uint32_t o_addr = tmem + 256 + tile * 128 + half * (D / 2) + lanes;
    const int pair = tile * 4 + (warp & 3);  // the two warps of the same rows
    const int HQ = p.H * G;
    const int t_row = row / G, g_row = row - t_row * G;  // token and head of this row in its tile
    const bool neg = p.qscale < 0.f;
    const bool sectors = ((reinterpret_cast<uintptr_t>(p.o) | (uintptr_t)p.o_stride * 2) & 31) == 0;
    int step = 0, items = 0;  // steps and items of this row tile so far
    bool ok = true;
    // The exchange of a step.  With one row tile the next step may begin while the other
    // thread still reads: two places in turn.  With two it begins with scores that wait
    // for both threads' weights.
    auto told = [&](int s, int which) -> float& {
      return S.half[C::kTiles == 2 ? which * (2 * kTileRows) + hrow
                                   : (s & 1) * (2 * kTileRows) + which * kTileRows + row];
    };
    for (int k = 0;; ++k) {
      Item it;
      it.id = -1;
      ok = ok && next_item(k, it);
      // a wait that ran out ends both warps of a pair at the same place
      if (lane == 0) S.fine[k & 1][pair][half] = ok;
      named_barrier(1 + pair, 64);
      if (!ok || !S.fine[k & 1][pair][half ^ 1] || it.id < 0) break;
      if (tile * per_tile >= it.tokens) continue;  // no rows in this tile
      const bool live = t_row < per_tile && tile * per_tile + t_row < it.tokens;
      const int token = it.first + tile * per_tile + t_row, head = it.h * G + g_row;
      int see_lo = 0, see_hi = 0x7fffffff;  // a row that is not written need not be masked
      if (live) {
        see_hi = it.len;
        if (p.range) {
          see_lo = max(0, p.range[2 * (int64_t)token]);
          see_hi = max(0, min(see_hi, p.range[2 * (int64_t)token + 1]));
        }
      }
      const int32_t* table = p.table + (int64_t)it.b * p.max_pages;
      const int nk = it.nk;
      float m = kNone, l = 0.f;
      uint32_t pages_ok = 0;
      for (int n = 0; n < nk; ++n, ++step) {
        const int buf = C::kTiles == 2 ? tile : step & 1, parity = (C::kTiles == 2 ? step : step >> 1) & 1;
        if ((n & 15) == 0) {
          const int pg = it.page0 + 2 * n + lane;
          const int32_t e = pg < it.page_end ? table[pg] : -1;
          pages_ok = __ballot_sync(0xffffffffu, e >= 0 && e < p.kv_slots);
        }
        const int k0 = (it.page0 + 2 * n + half) * kPageTokens;
        const bool there = pages_ok >> (2 * (n & 15) + half) & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full[buf], parity, p.status, p.wait_ns)) != 0;
        tc_fence_after();
        const uint32_t s_addr = tmem + buf * kKeys + half * kMine + lanes;
        const int lo = see_lo - k0, hi = see_hi - k0;
        const bool plain = !neg && __all_sync(0xffffffffu, lo <= 0 && hi >= kMine && there);
        // scores [c, c + 32) of this half; they are read twice, which takes half the
        // registers and next to no time.  (The roles share an instruction cache: of the
        // loops over them only the first is unrolled, with two row tiles, 316 -> 302 us at
        // eight prompts; with one tile that costs 4 %.)
        auto scores = [&](float(&x)[32], int c) {
          tc_ld32(x, s_addr + c);
          tc_wait_ld();
          tc_loaded(x);
          if (!plain) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              x[e] = neg ? -x[e] : x[e];
              if (c + e < lo || c + e >= hi || !there) x[e] = kNone;
            }
          }
        };
        float top[4] = {kNone, kNone, kNone, kNone};
#pragma unroll (C::kTiles == 2 ? 2 : 1)
        for (int c = 0; c < kMine; c += 32) {
          float x[32];
          scores(x, c);
#pragma unroll
          for (int e = 0; e < 32; e += 2) top[e >> 1 & 3] = fmaxf(fmaxf(top[e >> 1 & 3], x[e]), x[e + 1]);
        }
        // the row's other half; both then take the same decisions (a wait that ran out
        // is told as NaN, which no maximum is)
        const float mine = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        told(step, half) = ok ? mine : __int_as_float(0x7fffffff);
        named_barrier(1 + pair, 64);
        const float other = told(step, half ^ 1);
        ok = ok && !__any_sync(0xffffffffu, other != other);
        if (!ok) break;
        const float mt = fmaxf(mine, other) * qscale;
        const bool grow = mt - m > kLift<T> + kSlack<T>;  // not where both are -inf
        if (__any_sync(0xffffffffu, grow)) {
          const float to = mt - kLift<T>, f = !grow ? 1.f : far_off<T>(m) ? __int_as_float(0x7fffffff) : ex2(m - to);
          l *= f;
          if (grow) m = to;
          if (n > 0) {
            // the product before these weights has ended: with two tiles it came before
            // the scores just read
            bool done = true;
            if (C::kTiles == 1) done = __all_sync(0xffffffffu, mbar_wait(&S.pv_done, (step - 1) & 1, p.status, p.wait_ns)) != 0;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 2 && done; c += 32) {
              float o[32];
              tc_ld32(o, o_addr + c);
              tc_wait_ld();
              tc_loaded(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tc_st32(o_addr + c, o);
            }
            tc_wait_st();
          }
        }
        const float ref = m == kNone ? 0.f : m;
        const uint64_t q2 = ::tpk::pair(qscale, qscale), ref2 = ::tpk::pair(-ref, -ref);
        uint64_t sum[2] = {0, 0};
#pragma unroll 1
        for (int c = 0; c < kMine; c += 32) {
          float x[32];
          uint32_t w[16];
          scores(x, c);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 v = unpair(fma2(::tpk::pair(x[e], x[e + 1]), q2, ref2));
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], ::tpk::pair(v.x, v.y));
            w[e >> 1] = T::pack(v.x, v.y);
          }
          tc_st16(s_addr + (c >> 1), w);  // over scores of this half already used
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(c == 0 ? &S.p_half[buf] : &S.p_full[buf]);
        }
        const float2 both = unpair(add2(sum[0], sum[1]));
        l += both.x + both.y;
      }
      if (!ok) continue;
      // ---- the rows' results
      if (nk > 0) {
        named_barrier(1 + pair, 64);
        told(0, half) = l;
        named_barrier(1 + pair, 64);
        l += told(0, half ^ 1);
        if (far_off<T>(m)) l = __int_as_float(0x7fffffff);
        ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[tile], items++ & 1, p.status, p.wait_ns)) != 0;
        tc_fence_after();
      }
      const int64_t at = (int64_t)it.id * C::kRows + hrow;  // this part's row in the workspace
      const float inv = splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      // the fold does not use an empty part (by its sum: one of NaN scores has no maximum either)
      const bool write = live && ok && !(splits > 1 && l == 0.f);
      if (live && ok && half == 0) {
        if (splits > 1) {
          p.part_ml[2 * at] = m;
          p.part_ml[2 * at + 1] = l;
        } else {
          p.lse[(int64_t)token * HQ + head] = l == 0.f ? kNone : (m + log2f(l)) * kLn2;
        }
      }
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        __syncwarp();
        if (nk > 0) {
          tc_ld32(o, o_addr + c);
          tc_wait_ld();
          tc_loaded(o);
          if (c + 32 == D / 2) {
            tc_fence_before();
            mbar_arrive(&S.o_empty[tile]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        const int ch = half * (D / 2) + c;
        if (write && splits > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + ch);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else if (write) {
          uint16_t* dst = static_cast<uint16_t*>(p.o) + (int64_t)token * p.o_stride + (int64_t)head * D + ch;
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = T::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
          if (sectors) {  // whole 32-byte sectors
            store32(dst, w);
            store32(dst + 16, w + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<uint4*>(dst)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == C::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem);
  }
  // No copy is in flight when the block ends, whichever role gave up.  (A copy into a slot means
  // that the one before it there has landed.)
  if (tid < C::kSlots + 2) {
    uint64_t* const bar = tid < C::kSlots ? &S.full[tid] : tid == C::kSlots ? &S.tail : &S.q_full;
    const int n = tid < C::kSlots ? S.laps[tid] : tid == C::kSlots ? S.tails : S.loads;
    if (n > 0) mbar_wait(bar, (n - 1) & 1, p.status, p.wait_ns);
  }
}

// Joins the parts of a split launch, one warp per row of a tile group, which the group's record
// gives its query token; kJoined parts' values in flight.
constexpr int kJoined = 4;
template <typename T, int D, int kT>
__global__ void __launch_bounds__(256) tile_fold_kernel(const __grid_constant__ PagedParams p, int splits) {
  using C = TileCfg<D, kT>;
  const int lane = threadIdx.x & 31, per_tile = kTileRows / p.G;
  // 32 bits do: keys are split only where all items together are at most kTileBlocks
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = w % C::kRows, group = w / C::kRows, h = group % p.H;  // group: of tiles, and a head
  const int x = r % kTileRows / p.G, t = r / kTileRows * per_tile + x;
  auto at = [&](int k) { return (group * splits + k) * C::kRows + r; };
  wait_before();  // nothing is read before it
  // the group's query tokens; a part's (maximum, sum) a lane; the first parts' values
  const RunCut cut = p.cuts[group];
  float2 ml = make_float2(kNone, 0.f), v[kJoined][D / 64];
  if (lane < splits) ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at(lane));
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kJoined; ++j)
      if (k0 + j < splits)
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
          v[j][e] = *reinterpret_cast<const float2*>(p.part_o + (int64_t)at(k0 + j) * D + e * 64 + 2 * lane);
  };
  // (a record that a block which gave up did not write may hold anything)
  const int token = cut.first + t, head = h * p.G + r % kTileRows - x * p.G;
  if (x >= per_tile || t >= cut.count || (unsigned)cut.first >= (unsigned)p.n_q || token >= p.n_q) return;
  load(0);
  float M = ml.x;
  for (int k = lane + 32; k < splits; k += 32) M = fmaxf(M, p.part_ml[2 * at(k)]);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float L = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int k0 = 0; k0 < splits; k0 += kJoined) {
    if (k0 > 0) load(k0);
    if (k0 > 0 && (k0 & 31) == 0 && k0 + lane < splits)
      ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at(k0 + lane));
#pragma unroll
    for (int j = 0; j < kJoined; ++j) {
      if (k0 + j >= splits) break;
      const float m = __shfl_sync(0xffffffffu, ml.x, (k0 + j) & 31), l = __shfl_sync(0xffffffffu, ml.y, (k0 + j) & 31);
      if (l == 0.f) continue;
      const float f = exp2f(m - M);  // NaN where no part has a maximum: what sums there are are NaN
      L += f * l;
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        o[2 * e] += f * v[j][e].x;
        o[2 * e + 1] += f * v[j][e].y;
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + (int64_t)token * p.o_stride + (int64_t)head * D);
#pragma unroll
  for (int e = 0; e < D / 64; ++e) dst[e * 32 + lane] = T::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0) p.lse[(int64_t)token * p.H * p.G + head] = L == 0.f ? kNone : (M + log2f(L)) * kLn2;
}

int device_sms();

template <typename T, int D, int kT>
static cudaError_t launch_t(const PagedParams& p, int groups, int splits, cudaStream_t stream) {
  using C = TileCfg<D, kT>;
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(tile_kernel<T, D, kT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (e != cudaSuccess) return e;
  e = launch_early(tile_kernel<T, D, kT>, groups * p.H * splits, C::kThreads, C::kSmem, stream, p, splits);
  if (e != cudaSuccess || splits == 1) return e;
  // the fold's blocks may start while the last parts still run: they wait for them
  return launch_early(tile_fold_kernel<T, D, kT>, groups * p.H * (C::kRows / 8), 256, 0, stream, p, splits);
}

template <int D, int kT>
static cudaError_t launch_type(const PagedParams& p, int dtype, int groups, int splits, cudaStream_t stream) {
  return dtype == 0 ? launch_t<Bf16, D, kT>(p, groups, splits, stream) : launch_t<F16, D, kT>(p, groups, splits, stream);
}

cudaError_t launch_cross_tiles(const PagedParams& p, int D, int dtype, int tiles, int groups, int splits,
                               cudaStream_t stream) {
  if (D == 256) return launch_type<256, 1>(p, dtype, groups, splits, stream);
  if (D == 128)
    return tiles == 1 ? launch_type<128, 1>(p, dtype, groups, splits, stream)
                      : launch_type<128, 2>(p, dtype, groups, splits, stream);
  return tiles == 1 ? launch_type<64, 1>(p, dtype, groups, splits, stream)
                    : launch_type<64, 2>(p, dtype, groups, splits, stream);
}

}  // namespace tpk
