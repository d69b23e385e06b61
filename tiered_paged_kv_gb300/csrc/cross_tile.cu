// Cross attention of many query rows on the fifth-generation tensor cores.
//
// A thread block takes 128-row tiles of one (request, KV head), rows being packed
// (query token, head) pairs: two tiles for D <= 128, one for D = 256 or where the rows
// end.  The keys and values pass once, 128 tokens (two pages) at a time, through a ring
// of shared-memory slots filled by TMA.  Per key tile S = Q K^T goes to TMEM, one thread
// per row turns its 128 scores into weights (online softmax in base 2), writes them over
// S in the input type, and O += P V runs with P read from TMEM as the A operand.
//
// The steps are numbered so that the tensor core always has work while a softmax runs:
// step i uses score buffer i mod 2 and is (tile i mod 2, keys i / 2) with two tiles, or
// keys i with one; the issuing thread runs QK(0), QK(1), then PV(i), QK(i + 2), ...  The
// matrix instructions of one thread execute in order, so QK(i + 2) may overwrite the
// buffer that PV(i) reads its weights from.
//
// The reference maximum of a row moves only when the running maximum has grown by more
// than 2^8 (weights then stay below 256, exact in range for both types), so the pass that
// rescales O in TMEM is rare.  Weights are rounded once to the input type -- as the
// tensor core needs them beside V -- while their sum is kept unrounded in float32: the
// rounding of a weight is of the size of the output's own.
//
// Few query rows leave the device empty, so the keys can be split into `splits` parts
// per tile; parts leave (maximum, sum, O) in the workspace and a fold joins them in part
// order.  Bound: the tensor cores (4 D operations per score) and, for D = 64, the
// exponentials.
#include "paged.cuh"

namespace tpk {

constexpr float kNone = -__builtin_huge_valf();
constexpr float kSlack = 8.f;  // log2 of the largest weight
constexpr int kKeys = 128;     // tokens of a key tile
constexpr int kTileRows = 128;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct TileCfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;
  static constexpr int kRows = kTiles * kTileRows;
  static constexpr int kSlotChannels = D < 128 ? D : 128;
  static constexpr int kSlotBytes = kKeys * kSlotChannels * 2;
  static constexpr int kParts = D / kSlotChannels;  // slots per key (or value) tile
  static constexpr int kSlots = D == 64 ? 8 : 5;
  static constexpr int kQBytes = kTileRows * D * 2;  // one tile
  static constexpr int kSmem = 1024 + kTiles * kQBytes + kSlots * kSlotBytes;
  static constexpr int kThreads = kTiles * 128 + 64;
};

struct TileShared {
  uint64_t full[8], empty[8];
  uint64_t s_full[2], p_full[2];  // scores written, weights written (by score buffer)
  uint64_t pv_done[2], o_full[2]; // a product ended, the last one (by tile)
  uint64_t q_full, tail, drain;
  uint32_t tmem;
  int b, tile, clo, chi;
  int scan[12];
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
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory operand descriptor, 128-byte swizzle: 8-row groups of 1024 bytes are
// `stride` apart; 64-channel chunks `leading` apart (read only where the channels are
// not the reduced dimension).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(leading >> 4) << 16 | (uint64_t)(stride >> 4) << 32 |
         1ull << 46 | 2ull << 61;
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

__device__ __forceinline__ int tiles_of(const PagedParams& p, int b, int rows) {
  int first, count;
  request_rows(p, b, first, count);
  return (int)(((int64_t)count * p.G + rows - 1) / rows);
}

template <typename T, int D>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 1)
    tile_kernel(const __grid_constant__ PagedParams p, int splits) {
  using C = TileCfg<D>;
  constexpr int kSoft = C::kTiles * 128;  // softmax threads
  extern __shared__ uint8_t raw[];
  uint8_t* qs = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* slots = qs + C::kTiles * C::kQBytes;
  __shared__ TileShared S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x % splits;
  const int h = blockIdx.x / splits % p.H;
  const int want = blockIdx.x / splits / p.H;  // tile group among all requests'

  // ---- which request holds it
  const int each = (p.n_req + C::kThreads - 1) / C::kThreads;
  const int b0 = min(tid * each, p.n_req), b1 = min(b0 + each, p.n_req);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_of(p, b, C::kRows);
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  if (lane == 31) S.scan[warp] = inc;
  if (tid == 0) {
    S.b = -1;
    S.clo = 0x7fffffff;
    S.chi = 0;
#pragma unroll
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 128);
      mbar_init(&S.pv_done[i], 1);
      mbar_init(&S.o_full[i], 1);
    }
    mbar_init(&S.q_full, kSoft);
    mbar_init(&S.tail, 1);
    mbar_init(&S.drain, 1);
    fence_mbar_init();
  }
  __syncthreads();
  int before = inc - mine;
  for (int w = 0; w < warp; ++w) before += S.scan[w];
  if (want >= before && want < before + mine) {
    for (int b = b0; b < b1; ++b) {
      const int n = tiles_of(p, b, C::kRows);
      if (want < before + n) {
        S.b = b;
        S.tile = want - before;
        break;
      }
      before += n;
    }
  }
  __syncthreads();
  const int b = S.b;
  if (b < 0) return;  // past the last request's rows
  int first, count, tok_lo, tok_hi;
  request_rows(p, b, first, count);
  request_span(p, b, tok_lo, tok_hi);
  const int64_t row0 = (int64_t)S.tile * C::kRows;
  const int64_t rows = (int64_t)count * p.G - row0;  // of this block, if fewer than C::kRows
  const int nt = C::kTiles == 2 && rows > kTileRows ? 2 : 1;

  // ---- what each row sees, and what the block has to pass over
  int see_lo = 0, see_hi = 0, token = 0, head = 0;
  bool live = false;
  if (tid < kSoft) {
    live = tid < rows;
    if (live) {
      const int64_t i = row0 + tid;
      const int t = (int)(i / p.G);
      token = first + t;
      head = h * p.G + (int)(i - (int64_t)t * p.G);
      see_hi = tok_hi;
      if (p.range) {
        see_lo = max(0, p.range[2 * (int64_t)token]);
        see_hi = min(tok_hi, p.range[2 * (int64_t)token + 1]);
        if (see_hi > see_lo) {
          atomicMin(&S.clo, see_lo);
          atomicMax(&S.chi, see_hi);
        } else {
          see_lo = see_hi = 0;
        }
      }
    }
  }
  if (warp == kSoft / 32) tmem_alloc(&S.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int clo = p.range ? S.clo : 0, chi = p.range ? S.chi : tok_hi;
  int page0 = chi > clo ? clo >> 6 : 0;
  const int page_end = (chi + 63) >> 6;
  int nk = chi > clo ? (page_end - page0 + 1) >> 1 : 0;  // key tiles
  {
    const int k0 = (int)((int64_t)nk * part / splits), k1 = (int)((int64_t)nk * (part + 1) / splits);
    page0 += 2 * k0;
    nk = k1 - k0;
  }
  const int steps = nt * nk;
  const uint32_t tmem = S.tmem;
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  // the ring holds the key and value tiles in the order the tensor core takes them
  auto k_item = [&](int j) { return C::kParts * (nt == 2 ? 2 * j : (j == 0 ? 0 : 2 * j - 1)); };
  auto v_item = [&](int j) { return C::kParts * (nt == 2 ? 2 * j + 1 : (j < nk - 1 ? 2 * j + 2 : 2 * j + 1)); };

  if (warp == kSoft / 32) {
    // ------------------------------------------------------------ matrix issue
    if (lane == 0 && steps > 0) {
      constexpr bool bf16 = IsBf16<T>::value;
      constexpr uint32_t id_qk = instruction(bf16, false, kKeys);
      constexpr uint32_t id_pv = instruction(bf16, true, C::kSlotChannels);
      bool ok = mbar_wait(&S.q_full, 0, p.status, p.wait_ns);
      tc_fence_after();
      auto wait_item = [&](int item) {
        for (int c = 0; c < C::kParts && ok; ++c)
          ok = mbar_wait(&S.full[(item + c) % C::kSlots], ((item + c) / C::kSlots) & 1, p.status, p.wait_ns);
        tc_fence_after();
      };
      auto free_item = [&](int item) {
        for (int c = 0; c < C::kParts; ++c) tc_commit(&S.empty[(item + c) % C::kSlots]);
      };
      auto qk = [&](int i) {
        const int tile = nt == 2 ? i & 1 : 0, j = nt == 2 ? i >> 1 : i, item = k_item(j);
        if (tile == 0) wait_item(item);
        if (!ok) return;
        const uint32_t q = smem_u32(qs) + tile * C::kQBytes;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int part_of = c * 64 / C::kSlotChannels;
          const uint32_t k = smem_u32(slots) + (item + part_of) % C::kSlots * C::kSlotBytes +
                             (c * 64 % C::kSlotChannels) / 64 * (kKeys * 128);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            tc_mma_ss(tmem + (i & 1) * kKeys, operand(q + c * (kTileRows * 128) + x * 32, 16, 1024),
                      operand(k + x * 32, 16, 1024), id_qk, c > 0 || x > 0);
        }
        tc_commit(&S.s_full[i & 1]);
        if (nt == 1 || tile == 1) free_item(item);
      };
      qk(0);
      if (steps > 1) qk(1);
      for (int i = 0; i < steps && ok; ++i) {
        const int tile = nt == 2 ? i & 1 : 0, j = nt == 2 ? i >> 1 : i, item = v_item(j);
        ok = mbar_wait(&S.p_full[i & 1], (i >> 1) & 1, p.status, p.wait_ns);
        if (ok && tile == 0) wait_item(item);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::kParts; ++c) {
          const uint32_t v = smem_u32(slots) + (item + c) % C::kSlots * C::kSlotBytes;
#pragma unroll
          for (int x = 0; x < kKeys / 16; ++x)
            tc_mma_ts(tmem + 256 + tile * 128 + c * 128, tmem + (i & 1) * kKeys + x * 8,
                      operand(v + x * 2048, kKeys * 128, 1024), id_pv, j > 0 || x > 0);
        }
        tc_commit(&S.pv_done[tile]);
        if (j == nk - 1) tc_commit(&S.o_full[tile]);
        if (nt == 1 || tile == 1) free_item(item);
        if (i + 2 < steps) qk(i + 2);
      }
      tc_commit(&S.drain);
      mbar_wait(&S.drain, 0, p.status, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == kSoft / 32 + 1) {
    // ------------------------------------------------------------------ loader
    int item = 0;
    bool ok = true;
    int32_t near = 0, far = 0;  // table entries of this window of 16 key tiles, and of the one before
    int window = -1;
    int tails = 0;
    // one key (or value) tile: two pages, kParts slots
    auto load = [&](int j, bool values) {
      if (j / 16 > window) {
        window = j / 16;
        far = near;
        const int pg = page0 + 32 * window + lane;
        near = pg < page_end ? table[pg] : -1;
      }
      const int32_t from = j / 16 == window ? near : far;
      int64_t slot[2];
      bool there[2];
      int n = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        slot[x] = __shfl_sync(0xffffffffu, from, (2 * j + x) & 31);
        there[x] = slot[x] >= 0 && slot[x] < p.kv_slots;
        if (!there[x] && page0 + 2 * j + x < page_end && lane == 0) atomicOr(p.status, kStatusBadSlot);
        n += there[x];
      }
      const int k0 = (page0 + 2 * j) * kPageTokens;
      const bool clear = values && (n < 2 || k0 + kKeys > tok_hi);  // rows that must not be read as they are
      for (int c = 0; c < C::kParts && ok; ++c, ++item) {
        const int st = item % C::kSlots;
        if (item >= C::kSlots)
          ok = __all_sync(0xffffffffu, mbar_wait(&S.empty[st], (item / C::kSlots - 1) & 1, p.status, p.wait_ns));
        if (!ok) break;
        uint8_t* dst = slots + st * C::kSlotBytes;
        uint64_t* bar = clear ? &S.tail : &S.full[st];
        if (lane == 0) {
          if (n > 0) mbar_arrive_expect_tx(bar, n * (C::kSlotBytes / 2));
          else mbar_arrive(bar);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (there[x])
#pragma unroll
              for (int ch = 0; ch < C::kSlotChannels; ch += 64)
                tma_load_2d(dst + ch / 64 * (kKeys * 128) + x * (kPageTokens * 128), values ? &p.vmap : &p.kmap,
                            c * C::kSlotChannels + ch, (int)((slot[x] * p.H + h) * kPageTokens), bar);
        }
        __syncwarp();
        if (clear) {
          ok = __all_sync(0xffffffffu, mbar_wait(&S.tail, tails & 1, p.status, p.wait_ns));
          ++tails;
          for (int i = lane; i < kKeys * (C::kSlotChannels / 8); i += 32) {
            const int r = i / (C::kSlotChannels / 8), piece = i % (C::kSlotChannels / 8);
            if (!there[r >> 6] || k0 + r >= tok_hi)
              *reinterpret_cast<uint4*>(dst + (piece >> 3) * (kKeys * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.full[st]);
        }
      }
    };
    if (nt == 2) {
      for (int j = 0; j < nk && ok; ++j) {
        load(j, false);
        load(j, true);
      }
    } else {
      for (int j = 0; j < nk && ok; ++j) {
        if (j == 0) load(0, false);
        if (j + 1 < nk) load(j + 1, false);
        load(j, true);
      }
    }
    if (!ok)  // let the copies in flight land before the block ends
      for (int i = max(0, item - C::kSlots); i < item; ++i)
        mbar_wait(&S.full[i % C::kSlots], (i / C::kSlots) & 1, p.status, p.wait_ns);
  } else {
    // ----------------------------------------------------------------- softmax
    const int tile = warp >> 2;
    const float qscale = fabsf(p.qscale);  // its sign goes into q
    if (steps > 0) {
      const uint32_t flip = p.qscale < 0.f ? 0x80008000u : 0u;
      for (int i = tid; i < nt * kTileRows * (D / 8); i += kSoft) {
        const int r = i / (D / 8), piece = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          const int64_t x = row0 + r;
          const int t = (int)(x / p.G);
          v = *reinterpret_cast<const uint4*>(p.q + (int64_t)(first + t) * p.q_stride +
                                              (int64_t)(h * p.G + (int)(x - (int64_t)t * p.G)) * D + piece * 8);
          v.x ^= flip;
          v.y ^= flip;
          v.z ^= flip;
          v.w ^= flip;
        }
        const int rr = r & (kTileRows - 1);
        *reinterpret_cast<uint4*>(qs + (r >> 7) * C::kQBytes + (piece >> 3) * (kTileRows * 128) + rr * 128 +
                                  (((piece & 7) ^ (rr & 7)) << 4)) = v;
      }
      fence_async_smem();
      mbar_arrive(&S.q_full);
    }
    float m = kNone, l = 0.f;
    bool ok = true;
    uint32_t pages_ok = 0;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's TMEM rows
    const uint32_t o_addr = tmem + 256 + tile * 128 + lanes;
    const int n_mine = tile < nt ? nk : 0;
    for (int n = 0; n < n_mine && ok; ++n) {
      const int i = nt == 2 ? 2 * n + tile : n;
      if ((n & 15) == 0) {
        const int pg = page0 + 2 * n + lane;
        const int32_t e = pg < page_end ? table[pg] : -1;
        pages_ok = __ballot_sync(0xffffffffu, e >= 0 && e < p.kv_slots);
      }
      const int k0 = (page0 + 2 * n) * kPageTokens;
      const uint32_t halves = pages_ok >> (2 * (n & 15)) & 3;
      ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full[i & 1], (i >> 1) & 1, p.status, p.wait_ns));
      if (!ok) break;
      tc_fence_after();
      const uint32_t s_addr = tmem + (i & 1) * kKeys + lanes;
      float x[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) tc_ld32(x + c, s_addr + c);
      tc_wait_ld();
      tc_loaded(x);
      const int lo = see_lo - k0, hi = see_hi - k0;
      if (!__all_sync(0xffffffffu, lo <= 0 && hi >= kKeys && halves == 3)) {
#pragma unroll
        for (int c = 0; c < kKeys; ++c)
          if (c < lo || c >= hi || !(halves >> (c >> 6) & 1)) x[c] = kNone;
      }
      float top[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
      for (int c = 0; c < kKeys; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
      const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * qscale;
      const bool grow = mt > m + kSlack || (m == kNone && mt > kNone);
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? ex2(m - mt) : 1.f;
        l *= f;
        if (grow) m = mt;
        if (n > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&S.pv_done[tile], (n - 1) & 1, p.status, p.wait_ns));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
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
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float a = ex2(fmaf(x[c + e], qscale, -ref)), d = ex2(fmaf(x[c + e + 1], qscale, -ref));
          sum[e & 2] += a;
          sum[(e & 2) + 1] += d;
          w[e >> 1] = T::pack(a, d);
        }
        tc_st16(s_addr + (c >> 1), w);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&S.p_full[i & 1]);
    }
    // ---- the rows' results
    if (n_mine > 0 && ok) {
      ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[tile], 0, p.status, p.wait_ns));
      tc_fence_after();
    }
    if (ok && tile < nt) {
      const int HQ = p.H * p.G;
      const int64_t at = ((int64_t)blockIdx.x * C::kRows + tid);  // this part's row in the workspace
      const float inv = splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      if (live) {
        if (splits > 1) {
          p.part_ml[2 * at] = m;
          p.part_ml[2 * at + 1] = l;
        } else {
          p.lse[(int64_t)token * HQ + head] = l == 0.f ? kNone : (m + log2f(l)) * kLn2;
        }
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        __syncwarp();
        if (n_mine > 0) {
          tc_ld32(o, o_addr + c);
          tc_wait_ld();
          tc_loaded(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (!live) continue;
        if (splits > 1) {
          if (m == kNone) continue;  // the fold does not read an empty part
          float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (int64_t)token * p.o_stride +
                                                (int64_t)head * D + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(T::pack(o[8 * e] * inv, o[8 * e + 1] * inv), T::pack(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                T::pack(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                T::pack(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kSoft / 32) {
    tc_fence_after();
    tmem_dealloc(tmem);
  }
}

// Joins the parts of a split launch, one warp per row of a tile group.
template <typename T, int D>
__global__ void __launch_bounds__(256) tile_fold_kernel(const __grid_constant__ PagedParams p, int splits) {
  using C = TileCfg<D>;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = (int)(w % C::kRows);
  const int h = (int)(w / C::kRows % p.H);
  int want = (int)(w / C::kRows / p.H), b = 0;
  for (; b < p.n_req; ++b) {
    const int n = tiles_of(p, b, C::kRows);
    if (want < n) break;
    want -= n;
  }
  if (b == p.n_req) return;
  int first, count;
  request_rows(p, b, first, count);
  const int64_t i = (int64_t)want * C::kRows + r;
  if (i >= (int64_t)count * p.G) return;
  const int t = (int)(i / p.G), token = first + t, head = h * p.G + (int)(i - (int64_t)t * p.G);
  const int64_t group = w / C::kRows;  // (tile group, head)
  auto at = [&](int k) { return (group * splits + k) * C::kRows + r; };
  float M = kNone;
  for (int k = 0; k < splits; ++k) M = fmaxf(M, p.part_ml[2 * at(k)]);
  float L = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int k = 0; k < splits; ++k) {
    const float m = p.part_ml[2 * at(k)];
    if (m == kNone) continue;
    const float f = exp2f(m - M);
    L += f * p.part_ml[2 * at(k) + 1];
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      const float2 v = *reinterpret_cast<const float2*>(p.part_o + at(k) * D + e * 64 + 2 * lane);
      o[2 * e] += f * v.x;
      o[2 * e + 1] += f * v.y;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + (int64_t)token * p.o_stride + (int64_t)head * D);
#pragma unroll
  for (int e = 0; e < D / 64; ++e) dst[e * 32 + lane] = T::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0) p.lse[(int64_t)token * p.H * p.G + head] = L == 0.f ? kNone : (M + log2f(L)) * kLn2;
}

int device_sms();

template <typename T, int D>
static cudaError_t launch_t(const PagedParams& p, int groups, int splits, cudaStream_t stream) {
  using C = TileCfg<D>;
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(tile_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (e != cudaSuccess) return e;
  tile_kernel<T, D><<<groups * p.H * splits, C::kThreads, C::kSmem, stream>>>(p, splits);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  tile_fold_kernel<T, D><<<groups * p.H * (C::kRows / 8), 256, 0, stream>>>(p, splits);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_type(const PagedParams& p, int dtype, int groups, int splits, cudaStream_t stream) {
  return dtype == 0 ? launch_t<Bf16, D>(p, groups, splits, stream) : launch_t<F16, D>(p, groups, splits, stream);
}

int tile_rows(int D) { return D == 256 ? TileCfg<256>::kRows : TileCfg<128>::kRows; }

cudaError_t launch_cross_tiles(const PagedParams& p, int D, int dtype, int groups, int splits, cudaStream_t stream) {
  return D == 64    ? launch_type<64>(p, dtype, groups, splits, stream)
         : D == 128 ? launch_type<128>(p, dtype, groups, splits, stream)
                    : launch_type<256>(p, dtype, groups, splits, stream);
}

}  // namespace tpk
