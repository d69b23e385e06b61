// Host side of the calls over device-side lengths: argument validation, tensor maps
// and launches.  Lengths, tables and slot maps stay on the device, so what can be
// checked here is shapes, strides, alignment and sizes; the kernels clamp or skip the
// rest and report it in the device status word.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "paged.cuh"
#include "tpk.h"

namespace tpk {
void set_error(const char* msg);
int* device_status_word();
void* tensor_map_encoder();
uint64_t wait_limit_ns();
int stall_unit();
}  // namespace tpk

using namespace tpk;

namespace {

tpk_status fail(tpk_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_error(buf);
  return s;
}

tpk_status cuda_fail(cudaError_t e, const char* what) {
  return fail(TPK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Arrays of 4-byte (and one of 8-byte) elements, read as such; null passes.
template <typename... P>
bool aligned_to(size_t bytes, P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (bytes - 1)) == 0;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kMaxHeads = 1024, kMaxGroup = 128, kMaxTableRow = (1 << 25) - 1;

tpk_status check_paged(const tpk_paged_shape* s) {
  if (!s) return fail(TPK_ERR_INVALID, "shape is null");
  if (s->kv_heads < 1 || s->kv_heads > kMaxHeads) return fail(TPK_ERR_INVALID, "kv_heads %d out of [1, %d]", s->kv_heads, kMaxHeads);
  if (s->group < 1 || s->group > kMaxGroup) return fail(TPK_ERR_INVALID, "group %d out of [1, %d]", s->group, kMaxGroup);
  if (s->head_dim != 64 && s->head_dim != 128 && s->head_dim != 256)
    return fail(TPK_ERR_UNSUPPORTED, "head_dim %d (64, 128 or 256 supported)", s->head_dim);
  if (s->page_tokens != kPageTokens) return fail(TPK_ERR_UNSUPPORTED, "page_tokens %d (only 64 supported)", s->page_tokens);
  if (s->dtype != TPK_BF16 && s->dtype != TPK_F16) return fail(TPK_ERR_INVALID, "dtype %d", s->dtype);
  if (!std::isfinite(s->sm_scale)) return fail(TPK_ERR_INVALID, "sm_scale is not finite");
  if (s->kv_slots < 1) return fail(TPK_ERR_INVALID, "kv_slots %lld < 1", (long long)s->kv_slots);
  if (s->kv_slots > 0x7fffffffLL / ((int64_t)s->kv_heads * kPageTokens))
    return fail(TPK_ERR_UNSUPPORTED, "pool too large for one tensor map");
  return TPK_OK;
}

tpk_status check_stride(const char* what, int64_t stride, int64_t least) {
  if (stride < least) return fail(TPK_ERR_INVALID, "%s %lld < %lld", what, (long long)stride, (long long)least);
  if (stride % 8) return fail(TPK_ERR_INVALID, "%s %lld is not a multiple of 8 elements", what, (long long)stride);
  return TPK_OK;
}

// A tensor of 16-bit values with boxes of 64 channels and the 128-byte swizzle.
tpk_status make_map(CUtensorMap* map, int dtype, int rank, const void* base, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box) {
  typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  EncodeFn fn = reinterpret_cast<EncodeFn>(tensor_map_encoder());
  if (!fn) return fail(TPK_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = with_context([&] {
    return fn(map, dtype == TPK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
  return r == CUDA_SUCCESS ? TPK_OK : fail(TPK_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// The pools for the split kernel (whole: every channel in one box of kBoxRows rows), or for
// the row tiles (boxes of a page's rows and 64 channels).
tpk_status make_maps(PagedParams& p, const tpk_paged_shape* s, const void* k_pool, const void* v_pool, bool whole) {
  const cuuint64_t D = s->head_dim, rows = (cuuint64_t)s->kv_slots * s->kv_heads * kPageTokens;
  const cuuint64_t dims[3] = {whole ? 64 : D, rows, D / 64};
  const cuuint64_t strides[2] = {D * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)(whole ? kBoxRows : kPageTokens), (cuuint32_t)(D / 64)};
  const int rank = whole ? 3 : 2;
  const tpk_status st = make_map(&p.kmap, s->dtype, rank, k_pool, dims, strides, box);
  return st == TPK_OK ? make_map(&p.vmap, s->dtype, rank, v_pool, dims, strides, box) : st;
}

// Workspace of a split launch: the records of the runs to join, then the partials.
size_t split_ws_bytes(const tpk_paged_shape* s) {
  const size_t slots = 2 * (size_t)kPagedMaxBlocks * kRowTile;
  return align256(kPagedMaxBlocks * sizeof(RunCut)) + align256(2 * slots * 4) + slots * s->head_dim * 4;
}

void place_ws(PagedParams& p, void* ws) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.cuts = reinterpret_cast<RunCut*>(w);
  w += align256(kPagedMaxBlocks * sizeof(RunCut));
  p.part_ml = reinterpret_cast<float*>(w);
  w += align256(4 * (size_t)kPagedMaxBlocks * kRowTile * 4);
  p.part_o = reinterpret_cast<float*>(w);
}

// How cross attention of n_q tokens is cut.  groups = 0: the split kernel's runs.
// Otherwise row-tile items of one or two 128-row tiles: `groups` bounds them for one KV
// head (whole ones, and one per request that is not), `splits` parts of the keys fill
// the device where they are few.  The rules go by what the host knows (lengths are on
// the device): n_req, n_q and the table's width.
struct CrossPlan {
  int tiles;
  int64_t groups, splits;
  int64_t rows(const tpk_paged_shape* s) const {  // of all blocks
    return groups * s->kv_heads * splits * tiles * kTileRows;
  }
};
CrossPlan cross_plan(const tpk_paged_shape* s, int n_req, int n_q) {
  const int64_t H = s->kv_heads, per_tile = kTileRows / s->group;
  // The split kernel spreads single pages over the device, the tiles read a page once for
  // 128 rows.  It wins:
  // - with up to eight rows a request, its narrow form (1000 requests of a token, 250 states,
  //   8 heads of 64: 109 us against 261; 120 of 1500: 68 and 102; one of 100, 8 x 4 of 128:
  //   5.5 and 7.3; four of 1000: 11.2 and 12.2; sixteen of 2000: 26.0 and 27.7);
  // - with up to sixteen, where it need not cut runs or there are many items (19 of 600, 8 of
  //   64: 10.7 and 12.4; 64 of 500, 8 of 128: 33 and 38; 16 of 2000: 29.8 and 27.6; 1000 of
  //   250, 8 of 64: 153 and 263), at head size 256 not (100 of 100, 2 x 8: 18.6 and 15.4);
  // - with more, where it need not cut runs, tables are short and a wave of blocks takes
  //   them all, in runs of 8 rows, or of 16 below head size 256 (two requests of 32 tokens, 500
  //   states, 8 x 4 of 128: 10.5 and 13.3; one of 16, 250 states, 4 x 8 of 256: 8.1 and
  //   11.6; 16 of 16, 200 states, 8 x 2 of 64, 384 runs of 16: 8.5 and 9.7; of 32, 640 runs:
  //   15.2 and 10.0);
  // - with few runs (split_few).
  const bool wide = s->head_dim == 256;
  const int64_t rows = (int64_t)n_q * s->group, items = (n_q / per_tile + n_req) * H;
  auto runs = [&](int run_rows) { return (rows / run_rows + n_req) * H; };
  const int64_t wave = split_blocks(s->head_dim) * kTileBlocks;
  const bool whole = split_whole(true, n_req, n_req * H, s->max_pages);
  if (rows <= 8 * (int64_t)n_req || (!wide && rows <= 16 * (int64_t)n_req && (whole || items > 4 * kTileBlocks)) ||
      (whole && s->max_pages <= kWholePages && runs(wide ? 8 : kRowTile) <= wave) || split_few(runs(8), s->max_pages))
    return {0, 0, 1};
  // Two tiles share the keys and values and take about 1.5 times one tile's time, so one
  // is better where it needs at most 1.5 times the waves (four requests of 128 tokens,
  // 3000 states, 8 x 4 heads of 128: 34 us with one tile, 47 with two; sixteen of 128, 1000
  // states, 8 x 2 heads of 64: 25 and 20).  Requests count as equally long.
  const int64_t each = ((int64_t)n_q + n_req - 1) / n_req;
  auto waves = [&](int tiles) {
    const int64_t items = n_req * ((each + tiles * per_tile - 1) / (tiles * per_tile)) * H;
    return (items + kTileBlocks - 1) / kTileBlocks;
  };
  const int tiles = s->head_dim == 256 || 2 * waves(1) <= 3 * waves(2) ? 1 : 2;  // 256: TMEM holds one
  const int64_t groups = n_q / (tiles * per_tile) + n_req;
  const int64_t splits = std::min<int64_t>(kTileBlocks / (groups * H), (s->max_pages + 3) / 4);  // two key tiles a part
  return {tiles, groups, std::max<int64_t>(splits, 1)};
}

// Workspace of split row tiles: the groups' records (at most kTileBlocks), each row's maximum and
// sum, then its output.
constexpr size_t kGroupBytes = (kTileBlocks * sizeof(RunCut) + 255) / 256 * 256;
size_t tile_ws_bytes(const tpk_paged_shape* s, size_t rows) {
  return kGroupBytes + align256(rows * 8) + rows * s->head_dim * 4;
}

size_t cross_ws_bytes(const tpk_paged_shape* s, int n_req, int n_q) {
  const CrossPlan c = cross_plan(s, n_req, n_q);
  if (c.groups == 0) return split_ws_bytes(s);
  if (c.splits == 1) return 256;
  return tile_ws_bytes(s, (size_t)c.rows(s));
}

// An upper bound of that for all calls of the same shape with at most n_req requests and n_q
// tokens: which kernel takes a call does not go by size alone.  Row tiles are cut to at most
// kTileBlocks items, and one request with more than eight rows may take them.
size_t cross_ws_bound(const tpk_paged_shape* s, int n_req, int n_q) {
  if ((int64_t)n_q * s->group <= 8) return split_ws_bytes(s);
  const int64_t items = ((int64_t)n_q / (kTileRows / s->group) + n_req) * s->kv_heads;
  const int64_t splits = s->max_pages > 0 ? (s->max_pages + 3) / 4 : 1;
  const int64_t most = items < kTileBlocks && splits < kTileBlocks ? std::min<int64_t>(items * splits, kTileBlocks) : kTileBlocks;
  return std::max(split_ws_bytes(s), tile_ws_bytes(s, most * (s->head_dim == 256 ? 1 : 2) * kTileRows));
}

bool sized(const tpk_paged_shape* s, int n_req) {
  return s && n_req >= 1 && n_req <= kMaxPagedReq && (s->head_dim == 64 || s->head_dim == 128 || s->head_dim == 256);
}

tpk_status check_counts(const tpk_paged_shape* s, int n_req) {
  if (s->max_pages < 1 || s->max_pages > kMaxTableRow)
    return fail(TPK_ERR_INVALID, "max_pages %d out of [1, %d]", s->max_pages, kMaxTableRow);
  if (n_req < 1 || n_req > kMaxPagedReq) return fail(TPK_ERR_INVALID, "n_req %d out of [1, %d]", n_req, kMaxPagedReq);
  return TPK_OK;
}

// What both attention calls check and fill in.
tpk_status begin_attention(PagedParams& p, const tpk_paged_shape* s, int n_req, const void* q, int64_t q_stride,
                           const void* k_pool, const void* v_pool, const int32_t* page_table, const int32_t* n_tokens,
                           void* o, int64_t o_stride, float* lse, void* ws, size_t ws_bytes, size_t need) {
  tpk_status st = check_counts(s, n_req);
  if (st != TPK_OK) return st;
  if (!q || !k_pool || !v_pool || !page_table || !n_tokens || !o || !lse || !ws)
    return fail(TPK_ERR_INVALID, "null pointer argument");
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(o) || !aligned16(ws))
    return fail(TPK_ERR_INVALID, "q, pools, o and ws must be 16-byte aligned");
  if (!aligned_to(4, page_table, n_tokens, lse)) return fail(TPK_ERR_INVALID, "page_table, n_tokens and lse must be 4-byte aligned");
  const int64_t row = (int64_t)s->kv_heads * s->group * s->head_dim;
  st = check_stride("q_stride", q_stride, row);
  if (st == TPK_OK) st = check_stride("o_stride", o_stride, row);
  if (st != TPK_OK) return st;
  if (ws_bytes < need) return fail(TPK_ERR_NOMEM, "workspace %zu bytes < %zu required", ws_bytes, need);
  std::memset(&p, 0, sizeof p);
  p.status = device_status_word();
  if (!p.status) return fail(TPK_ERR_CUDA, "cannot resolve the device status word");
  p.q = static_cast<const uint16_t*>(q);
  p.o = o;
  p.lse = lse;
  p.table = page_table;
  p.lens = n_tokens;
  p.q_stride = q_stride;
  p.o_stride = o_stride;
  p.kv_slots = s->kv_slots;
  p.wait_ns = wait_limit_ns();
  p.stall_unit = stall_unit();
  const float scale = s->sm_scale == 0.f ? 1.f / std::sqrt((float)s->head_dim) : s->sm_scale;
  p.qscale = scale * kLog2e;
  p.n_req = n_req;
  p.max_pages = s->max_pages;
  p.H = s->kv_heads;
  p.G = s->group;
  return TPK_OK;
}

}  // namespace

extern "C" {

tpk_status tpk_kv_tables_update(int n_req, int max_pages, const int32_t* len_old, const int32_t* len_new,
                                int32_t* page_table, int32_t* free_slots, int free_cap, const int32_t* n_free_in,
                                int32_t* n_free_out, int32_t* len_out, int32_t* granted, int32_t* tok_off,
                                int64_t* slot_map, int32_t* positions, int32_t* token_req, int max_tokens,
                                tpk_stream_t stream) {
  if (n_req < 1 || n_req > kMaxPagedReq) return fail(TPK_ERR_INVALID, "n_req %d out of [1, %d]", n_req, kMaxPagedReq);
  if (max_pages < 1 || max_pages > kMaxTableRow || (int64_t)n_req * max_pages > 0x7fffffffLL)
    return fail(TPK_ERR_INVALID, "page table of %d x %d entries", n_req, max_pages);
  if (free_cap < 0) return fail(TPK_ERR_INVALID, "free_cap %d < 0", free_cap);
  if (free_cap > 0x7fffffff - n_req * max_pages) return fail(TPK_ERR_INVALID, "free_cap %d too large", free_cap);
  if (max_tokens < 0 || max_tokens > 0x7fffffff - 16384) return fail(TPK_ERR_INVALID, "max_tokens %d", max_tokens);
  if (!len_old || !len_new || !page_table || !n_free_in || !n_free_out || !len_out || !granted || !tok_off ||
      (free_cap > 0 && !free_slots) || (max_tokens > 0 && (!slot_map || !positions || !token_req)))
    return fail(TPK_ERR_INVALID, "null pointer argument");
  if (!aligned_to(4, len_old, len_new, page_table, free_slots, n_free_in, n_free_out, len_out, granted, tok_off, positions, token_req) ||
      !aligned_to(8, slot_map))
    return fail(TPK_ERR_INVALID, "an array is not aligned to its elements");
  TablesParams p;
  p.len_old = len_old;
  p.len_new = len_new;
  p.page_table = page_table;
  p.free_slots = free_slots;
  p.n_free_in = n_free_in;
  p.n_free_out = n_free_out;
  p.len_out = len_out;
  p.granted = granted;
  p.tok_off = tok_off;
  p.slot_map = slot_map;
  p.positions = positions;
  p.token_req = token_req;
  p.status = device_status_word();
  if (!p.status) return fail(TPK_ERR_CUDA, "cannot resolve the device status word");
  p.n_req = n_req;
  p.max_pages = max_pages;
  p.free_cap = free_cap;
  p.max_tokens = max_tokens;
  const cudaError_t e = launch_tables(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TPK_OK : cuda_fail(e, "tables launch");
}

tpk_status tpk_kv_rope_append(const tpk_paged_shape* shape, int n_tokens, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* positions, int n_axes, const uint8_t* axis_of, const float* inv_freq,
                              int rot_dim, int interleaved, const int64_t* slot_map, void* q_out,
                              int64_t q_out_stride, void* k_pool, void* v_pool, tpk_stream_t stream) {
  tpk_status st = check_paged(shape);
  if (st != TPK_OK) return st;
  const int H = shape->kv_heads, HQ = H * shape->group, D = shape->head_dim;
  if (n_tokens < 0) return fail(TPK_ERR_INVALID, "n_tokens %d < 0", n_tokens);
  if (rot_dim < 0 || rot_dim > D || rot_dim % 16) return fail(TPK_ERR_INVALID, "rot_dim %d (a multiple of 16 up to %d)", rot_dim, D);
  if (interleaved != 0 && interleaved != 1) return fail(TPK_ERR_INVALID, "interleaved %d (0 or 1)", interleaved);
  const bool none = n_tokens == 0;  // empty rows have no address
  const bool queries = q || q_out, keys = (k || v || k_pool || v_pool) && !(none && !k && !v && k_pool && v_pool);
  if (queries && !(q && q_out)) return fail(TPK_ERR_INVALID, "q and q_out go together");
  if (keys && !(k && v && k_pool && v_pool)) return fail(TPK_ERR_INVALID, "k, v and both pools go together");
  if (!queries && !keys && !none) return fail(TPK_ERR_INVALID, "nothing to rotate or store");
  if (keys && !slot_map && !none) return fail(TPK_ERR_INVALID, "null slot_map");
  if (rot_dim > 0) {
    if ((!positions && !none) || !inv_freq) return fail(TPK_ERR_INVALID, "null positions or inv_freq");
    if (n_axes < 1 || n_axes > 4) return fail(TPK_ERR_INVALID, "n_axes %d out of [1, 4]", n_axes);
  }
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) || !aligned16(k_pool) || !aligned16(v_pool))
    return fail(TPK_ERR_INVALID, "q, k, v, q_out and pools must be 16-byte aligned");
  if (!aligned_to(4, positions, inv_freq) || !aligned_to(8, slot_map))
    return fail(TPK_ERR_INVALID, "positions, inv_freq or slot_map is not aligned to its elements");
  if (queries) {
    st = check_stride("q_stride", q_stride, (int64_t)HQ * D);
    if (st == TPK_OK) st = check_stride("q_out_stride", q_out_stride, (int64_t)HQ * D);
    if (st != TPK_OK) return st;
    if (q == q_out && q_stride != q_out_stride) return fail(TPK_ERR_INVALID, "q_out is q with another stride");
  }
  if (keys) {
    st = check_stride("k_stride", k_stride, (int64_t)H * D);
    if (st == TPK_OK) st = check_stride("v_stride", v_stride, (int64_t)H * D);
    if (st != TPK_OK) return st;
  }
  RopeParams p;
  std::memset(&p, 0, sizeof p);
  for (int j = 0; j < rot_dim / 2; ++j) {
    p.axis_of[j] = axis_of ? axis_of[j] : 0;
    if (p.axis_of[j] >= n_axes) return fail(TPK_ERR_INVALID, "axis_of[%d] = %d of %d axes", j, p.axis_of[j], n_axes);
  }
  if (none) return TPK_OK;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_pool = static_cast<uint16_t*>(k_pool);
  p.v_pool = static_cast<uint16_t*>(v_pool);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.slot_map = slot_map;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.slot_limit = shape->kv_slots * kPageTokens;
  p.status = device_status_word();
  if (!p.status) return fail(TPK_ERR_CUDA, "cannot resolve the device status word");
  p.n_tokens = n_tokens;
  p.H = H;
  p.HQ = queries ? HQ : 0;
  p.D = D;
  p.rot = rot_dim;
  const cudaError_t e = launch_rope(p, shape->dtype, interleaved, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TPK_OK : cuda_fail(e, "rotary store launch");
}

size_t tpk_decode_paged_workspace_bytes(const tpk_paged_shape* shape, int n_req) {
  return sized(shape, n_req) ? split_ws_bytes(shape) : 0;
}

tpk_status tpk_decode_attn_paged(const tpk_paged_shape* shape, int n_req, const void* q, int64_t q_stride,
                                 const void* k_pool, const void* v_pool, const int32_t* page_table,
                                 const int32_t* n_tokens, const int32_t* tok_begin, void* o, int64_t o_stride,
                                 int o_f32, float* lse, void* ws, size_t ws_bytes, tpk_stream_t stream) {
  tpk_status st = check_paged(shape);
  if (st != TPK_OK) return st;
  if (o_f32 != 0 && o_f32 != 1) return fail(TPK_ERR_INVALID, "o_f32 %d (0 or 1)", o_f32);
  if (!aligned_to(4, tok_begin)) return fail(TPK_ERR_INVALID, "tok_begin must be 4-byte aligned");
  PagedParams p;
  st = begin_attention(p, shape, n_req, q, q_stride, k_pool, v_pool, page_table, n_tokens, o, o_stride, lse, ws, ws_bytes,
                       tpk_decode_paged_workspace_bytes(shape, n_req));
  if (st == TPK_OK) st = make_maps(p, shape, k_pool, v_pool, true);
  if (st != TPK_OK) return st;
  place_ws(p, ws);
  p.begin = tok_begin;
  p.o_f32 = o_f32;
  p.n_q = n_req;
  const cudaError_t e = launch_paged_split(p, shape->head_dim, shape->dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TPK_OK : cuda_fail(e, "paged decode launch");
}

size_t tpk_cross_paged_workspace_bytes(const tpk_paged_shape* shape, int n_req, int n_q) {
  return sized(shape, n_req) && n_q >= 0 && shape->kv_heads > 0 && shape->group > 0 && shape->group <= kMaxGroup ? cross_ws_bound(shape, n_req, n_q) : 0;
}

tpk_status tpk_cross_attn_paged(const tpk_paged_shape* shape, int n_req, int n_q, const void* q, int64_t q_stride,
                                const int32_t* q_off, const void* k_pool, const void* v_pool,
                                const int32_t* page_table, const int32_t* n_tokens, const int32_t* kv_range, void* o,
                                int64_t o_stride, float* lse, void* ws, size_t ws_bytes, tpk_stream_t stream) {
  tpk_status st = check_paged(shape);
  if (st != TPK_OK) return st;
  if (n_q < 0 || (int64_t)n_q * shape->kv_heads * shape->group > 0x7fffffffLL)
    return fail(TPK_ERR_INVALID, "n_q %d (at most 2^31 query rows)", n_q);
  if (!q_off) return fail(TPK_ERR_INVALID, "null pointer argument");
  if (!aligned_to(4, q_off, kv_range)) return fail(TPK_ERR_INVALID, "q_off and kv_range must be 4-byte aligned");
  if (n_q == 0) return check_counts(shape, n_req);  // empty rows have no address
  PagedParams p;
  st = begin_attention(p, shape, n_req, q, q_stride, k_pool, v_pool, page_table, n_tokens, o, o_stride, lse, ws, ws_bytes,
                       sized(shape, n_req) ? cross_ws_bytes(shape, n_req, n_q) : 0);
  if (st != TPK_OK) return st;
  p.q_off = q_off;
  p.range = kv_range;
  p.n_q = n_q;
  const CrossPlan plan = cross_plan(shape, n_req, n_q);
  st = make_maps(p, shape, k_pool, v_pool, plan.groups == 0);
  if (st != TPK_OK) return st;
  cudaError_t e;
  if (plan.groups == 0) {
    place_ws(p, ws);
    e = launch_paged_split(p, shape->head_dim, shape->dtype, reinterpret_cast<cudaStream_t>(stream));
  } else {
    const int64_t rows = plan.rows(shape);
    if (rows > 0x7fffffffLL) return fail(TPK_ERR_UNSUPPORTED, "too many query rows");
    const cuuint64_t dims[3] = {(cuuint64_t)shape->head_dim, (cuuint64_t)shape->kv_heads * shape->group, (cuuint64_t)n_q};
    const cuuint64_t strides[2] = {(cuuint64_t)shape->head_dim * 2, (cuuint64_t)q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)shape->group, (cuuint32_t)(kTileRows / shape->group)};
    st = make_map(&p.qmap, shape->dtype, 3, q, dims, strides, box);
    if (st != TPK_OK) return st;
    p.cuts = static_cast<RunCut*>(ws);
    p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kGroupBytes);
    p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kGroupBytes + align256((size_t)rows * 8));
    e = launch_cross_tiles(p, shape->head_dim, shape->dtype, plan.tiles, (int)plan.groups, (int)plan.splits,
                           reinterpret_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? TPK_OK : cuda_fail(e, "cross attention launch");
}

}  // extern "C"
