// What the kernels over device-side lengths share: the launch parameters, the two
// 16-bit types, the warp-level matrix and shared-memory instructions as inline PTX.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace tpk {

constexpr int kMaxPagedReq = 4096;

// ------------------------------------------------------------------ tables
struct TablesParams {
  const int32_t* len_old;
  const int32_t* len_new;
  int32_t* page_table;
  int32_t* free_slots;
  const int32_t* n_free_in;
  int32_t* n_free_out;
  int32_t* len_out;
  int32_t* granted;
  int32_t* tok_off;
  int64_t* slot_map;
  int32_t* positions;
  int32_t* token_req;
  int* status;
  int n_req, max_pages, free_cap, max_tokens;
};
cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream);

// ------------------------------------------------------------ rotary store
struct RopeParams {
  const uint16_t* q;  // null: no queries
  const uint16_t* k;  // null: no keys and values
  const uint16_t* v;
  uint16_t* q_out;
  uint16_t* k_pool;
  uint16_t* v_pool;
  const int32_t* positions;
  const float* inv_freq;
  const int64_t* slot_map;  // null: every row is live
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int64_t slot_limit;  // kv_slots * 64
  int* status;
  int n_tokens, H, HQ, D, rot;
  uint8_t axis_of[128];
};
cudaError_t launch_rope(const RopeParams& p, int dtype, int interleaved, cudaStream_t stream);

// --------------------------------------------------------------- attention
constexpr int kBoxRows = 16;  // rows of a page in one copy of the split kernel: one warp's
// What a block records for the join of a run that crosses its range, or of a group of row tiles
// whose keys are split.
struct __align__(16) RunCut {
  int first, count;  // the request's query rows; the group's
  int h, tile;       // the run's KV head, and its number within the request's rows
  int parts;         // blocks that hold a piece of it; 0: no such run
};
struct PagedParams {
  // pools with the 128-byte swizzle.  Row tiles: [slot * H * 64][D], boxes of 64 rows x 64
  // channels; split kernel: [D / 64][slot * H * 64][64], boxes of all channels of kBoxRows rows
  CUtensorMap kmap;
  CUtensorMap vmap;
  CUtensorMap qmap;  // row tiles only: q as [n_q][H * G][D], boxes of 64 channels of a KV head's rows in a tile
  const uint16_t* q;
  void* o;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* begin;  // decode: first token attended, or null
  const int32_t* q_off;  // cross: where each request's query rows begin; null: decode
  const int32_t* range;  // cross: [n_q][2] or null
  RunCut* cuts;          // workspace: of each block, or group of row tiles
  float* part_ml;        // workspace: [slot][16] running maximum, then [slot][16] sum
  float* part_o;         // workspace: [slot][16][D], not normalised
  int* status;
  int64_t q_stride, o_stride, kv_slots;
  uint64_t wait_ns;
  float qscale;  // sm_scale * log2(e)
  int n_req, n_q, max_pages, H, G, o_f32;
  int run_rows;  // query rows of a run, 8 or 16 (set at launch)
  int whole;     // a block per run (set at launch)
  int stall_unit;  // test hook: this block's first page, or key tile, is neither copied nor signalled (-1: none)
};

constexpr int kTileBlocks = 152;  // SMs of the device: blocks a launch over row tiles aims at
constexpr int kPagedMaxBlocks = 512;  // blocks of a split launch; each owns two partial slots
constexpr int kRowTile = 16;          // query rows of a split run, at most
cudaError_t launch_paged_split(PagedParams& p, int D, int dtype, cudaStream_t stream);

constexpr int split_blocks(int D) { return D == 256 ? 1 : D == 128 ? 2 : 3; }  // resident per SM
constexpr int kScanned = 128;  // requests that one warp numbers: lane i has 4 i .. 4 i + 3
// Short histories are not split: a block per run walks its pages in less time than the
// numbering and the join take (one request of 4 pages, 8 x 8 heads of 128: 6.2 us whole, 9.1
// split; of 8: 8.1 and 9.1; of 12: 10.2 and 9.2).  With a run for every SM the device is
// busy either way, and splitting only costs (16 requests of 32 pages: 25.8 and 31.6); but
// the lengths are not known here, and one long history among short ones must not be left
// to one block for longer than that.  Cross attention counts one run a request and head, and
// finds a block's run by a warp's scan.
constexpr int kWholePages = 8, kWholePagesBusy = 32, kBusyRuns = 128;
inline bool split_whole(bool cross, int n_req, int64_t runs, int max_pages) {
  return max_pages <= (runs >= kBusyRuns ? kWholePagesBusy : kWholePages) && (!cross || n_req <= kScanned);
}
// Few runs of 8 rows, the split kernel's even where they are more than a request (one request of
// 16 rows, 3000 states, 8 heads of 128: 11.7 us, 14.6 as row tiles; 4 heads of 256: 11.6 and
// 18.2; of 64 rows, 36 runs: 17.6 and 20.2; of 128 rows, 8 heads of 128, 72 runs: 17.3 and 15.3;
// of 64 rows, 20,000 states, 4 heads of 256, 74 (page, run) units per SM: 56 and 52).
inline bool split_few(int64_t runs, int max_pages) { return runs <= 64 && runs * max_pages <= 50 * kTileBlocks; }
// Runs of 8 rather than 16 rows read pages twice, with less work on each: for as long as
// the pages stay in L2 (decode of 16 heads a group: 1000 tokens, 8 KV heads of 256, 10.8 us
// against 14.3 in runs of 16; 5000: 16.7 and 18.2; 20,000, 160 MB: 48 and 43).
inline bool read_twice(int64_t runs, int max_pages, int D) {
  return split_few(runs, max_pages) && runs * max_pages / 2 * (kPageTokens * 4 * D) <= 100 << 20;
}

constexpr int kTileRows = 128;    // query rows of a tile; a block takes `tiles` (1 or 2) of them
cudaError_t launch_cross_tiles(const PagedParams& p, int D, int dtype, int tiles, int groups, int splits,
                               cudaStream_t stream);

// ------------------------------------------------------------------- types
// kWeightBits: weights, at most 1, enter the product with the values times 2^kWeightBits.  float16
// steps by 2^-24 at its lower end, and many weights below that may count together: scaled by 2^15
// they fill its range (largest value 65,504).  bfloat16 has float32's range and needs no scale.
struct Bf16 {
  static constexpr int kWeightBits = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
struct F16 {
  static constexpr int kWeightBits = 15;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values, two of a row a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// One lane of a converged warp, which the compiler then knows to be alone.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(smem_dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// The kernels of a step start while the one before in the stream still ends (launch_early), and
// wait here for its results before they read or write anything.  Every block waits, whether it
// has work or not: a launch must not end before the one it waits for.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next launch start.  It may read what this one reads or writes only after its own wait:
// this launch's wait shows the results before it to this launch alone.
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Request b's attended tokens [lo, hi), cut into what its table row can hold.
__device__ __forceinline__ void request_span(const PagedParams& p, int b, int& lo, int& hi) {
  const int cap = p.max_pages * 64;
  const int n = p.lens[b];
  hi = min(max(n, 0), cap);
  lo = 0;
  bool bad = n != hi;
  if (p.begin) {
    const int a = p.begin[b];
    lo = min(max(a, 0), cap);
    bad |= a != lo;
  }
  if (bad) atomicOr(p.status, kStatusBadSlot);
}

// Request b's query rows: tokens [first, first + count) of q.
__device__ __forceinline__ void request_rows(const PagedParams& p, int b, int& first, int& count) {
  if (!p.q_off) {
    first = b;
    count = 1;
    return;
  }
  first = min(max(p.q_off[b], 0), p.n_q);
  count = max(min(max(p.q_off[b + 1], 0), p.n_q) - first, 0);
}

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tpk
