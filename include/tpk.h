/*
 * tpk -- split-tier paged decode attention for GB300 (sm_103a).  C ABI.
 *
 * One decode step attends the G query rows of each KV head over a long paged
 * history held in two tiers (pages by their titles: "ActiveKV", section "The
 * idea"; "SYCL", sections "Attention that reads 8-bit history" and "A merge that
 * joins the tiers"; "model quantization", section "An 8-bit page format shaped
 * for its kernel"):
 *   - a recent tier of BF16 pages, attended exactly;
 *   - an older tier of 8-bit page records read directly, never expanded;
 *   - per-tier partials (output o, log-sum-exp lse) folded by an exact FP32 merge.
 *
 * Conventions shared by every call
 * --------------------------------
 * Ownership  The caller owns every buffer.  The library allocates no device
 *            memory; the multi-request call takes a caller-provided workspace.
 * Pointers   "dev" pointers are device memory of the current device; "host"
 *            pointers are read on the host before the call returns.  Device
 *            pointers must be 16-byte aligned.
 * Streams    Every call is asynchronous on `stream` (a cudaStream_t; NULL is the
 *            legacy default stream).
 * Errors     Argument errors are detected on the host before any launch and
 *            returned as a status; nothing is launched then.  Launch failures
 *            map to TPK_ERR_CUDA.  Page-table entries outside the pool sizes
 *            given in tpk_shape are skipped by the kernels (that page then
 *            contributes nothing) and recorded in a device status word read by
 *            tpk_get_device_status.  The library never aborts or traps.
 *            tpk_last_error_string describes the last failure on this thread.
 * Layouts    BF16 pools:  [slot][kv_heads][64][256] bfloat16, K and V separate.
 *            8-bit pool:  record (slot, h) at byte (slot * kv_heads + h) * 35072.
 *            q:           [rows = kv_heads * group][256] bfloat16 (per request);
 *                         query row j belongs to KV head j / group.
 *            o:           float32 [rows][256], normalised (sum of weights 1).
 *            lse:         float32 [rows], natural log of sum exp(sm_scale q.k).
 * Empty      An empty token or page range yields lse = -inf and o = 0, the valid
 *            empty partial; a merge never reads the o of a -inf partial.
 * Contexts   Per device the library resolves once, on first use, the device
 *            addresses of its status word and static scratch, its kernels'
 *            shared-memory limits and its constant tables; they belong to the
 *            device's primary context.  Do not call cudaDeviceReset (or otherwise
 *            end that context) between calls of the library in one process.
 */
#ifndef TPK_H
#define TPK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* tpk_stream_t; /* identical to cudaStream_t */

typedef enum {
  TPK_OK = 0,
  TPK_ERR_INVALID = 1,     /* bad argument (null pointer, bad range, misalignment, too small buffer) */
  TPK_ERR_UNSUPPORTED = 2, /* shape outside what the kernels implement */
  TPK_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed */
  TPK_ERR_BOUNDS = 4,      /* a kernel met a page-table entry outside the pool */
  TPK_ERR_NOMEM = 5,       /* a caller-provided buffer is smaller than required */
  TPK_ERR_TIMEOUT = 6,     /* a bounded device-side wait gave up */
  TPK_ERR_FORMAT = 7       /* a kernel met a malformed 13-bit record */
} tpk_status;

/* Which dot-product engine the decode kernels use. */
enum { TPK_IMPL_DEFAULT = 0, TPK_IMPL_SIMT = 1, TPK_IMPL_TENSOR = 2 };

/* Bytes of one 8-bit page-head record:
 *   u8   kc[64][256]   key codes, token-major          offset 0
 *   u8   vc[256][64]   value codes, channel-major      offset 16384
 *   f32  ks_chan[256]  key channel scale s_c           offset 32768
 *   f32  ks_tok[64]    key per-token factor r_t        offset 33792
 *   f32  vs_chan[256]  value channel scale u_c         offset 34048
 * Position swizzles (the format is shaped for the kernel that reads it):
 *   key code (t, c)   at byte t*256 + (c XOR 64*(t mod 2))
 *   value code (c, t) at byte c*64 + (t XOR 32*((c/2) mod 2))
 *   s_c               at float (c XOR 8*((c/32) mod 2))
 * A code c in [-127, 127] is stored as the byte c + 128 (offset binary), so
 * the tensor-core kernel widens it to f16 with one byte permute.
 * Dequantised: k_tc = kc_tc * s_c * r_t and v_tc = vc_tc * u_c. */
#define TPK_RECORD_BYTES 35072

typedef struct {
  int kv_heads;      /* H >= 1 */
  int group;         /* G query rows per KV head; must be 8 */
  int head_dim;      /* must be 256 */
  int page_tokens;   /* must be 64 */
  float sm_scale;    /* softmax scale; 0 selects 1/sqrt(head_dim) (the only value supported) */
  int impl;          /* TPK_IMPL_* */
  int64_t kv_slots;  /* slots in the BF16 pools (bounds for page_table entries); 0 = unchecked,
                        allowed only with TPK_IMPL_SIMT: the tensor-core kernel reads the BF16
                        pools through TMA tensor maps that need the pool size */
  int64_t rec_slots; /* slots in the 8-bit pool (bounds for page_table8 entries); 0 = unchecked */
  int int_query;     /* 0 (default): the 8-bit tier's QK uses the query in floating point.
                        1: the integer-query variant ("SYCL", "Attention that reads 8-bit
                        history": the integer query cache): per record and query row the
                        folded query q'_c = q_c s_c is coded as qi_c = rint(q'_c * (127 / m)),
                        m = max_c |q'_c| over the 256 channels, float32 steps with correctly
                        rounded divisions, half to even; the score is
                        (m / 127) * r_t * sum_c qi_c kc_tc, the sum exact.  This changes the
                        result (the query is coded to 8 bits); the exact tier is unaffected.
                        Tensor-core kernel only (TPK_IMPL_SIMT gives TPK_ERR_UNSUPPORTED). */
} tpk_shape;

const char* tpk_version(void);
const char* tpk_last_error_string(void);

/*
 * Page conversion ("model quantization", section "An 8-bit page format shaped for
 * its kernel").  For each of n_pages pages and each KV head h, read the BF16 page
 * (src_slots[i], h) of k_pool / v_pool and write record (dst_slots[i], h) of
 * rec_pool:
 *   key channel scale  s_c = sqrt(RMS_t k_tc), normalised by the geometric mean so
 *                      prod_c s_c = 1, clamped to [2^-14, 2^14], rounded to float32
 *                      with compensated rounding (the running log-error of the
 *                      product is kept nearest zero);
 *   key token factor   r_t = max_c |k_tc / s_c| / 127;
 *   value scale        u_c = max_t |v_tc| / 127;
 *   codes              kc = rint((k / s_c) / r_t), vc = rint(v / u_c), clamped to
 *                      +-127, with IEEE float32 divisions and half-to-even rint;
 *                      a zero factor gives zero codes.
 * src_slots, dst_slots: dev int32[n_pages].  k_pool, v_pool: dev BF16 pools.
 * rec_pool: dev, 16-byte aligned.  Pages may be converted in any order; distinct
 * dst_slots must not alias.  n_pages == 0 is a no-op.
 */
tpk_status tpk_kv_quantize_pages(const tpk_shape* shape, const void* k_pool, const void* v_pool,
                                 const int32_t* src_slots, const int32_t* dst_slots, int n_pages,
                                 void* rec_pool, tpk_stream_t stream);

/*
 * As tpk_kv_quantize_pages, but with all three scale arrays given (dev float32
 * ks_chan[n_pages][H][256], ks_tok[n_pages][H][64], vs_chan[n_pages][H][256]);
 * only the codes are computed, and the given scales are copied into the records.
 * Used to check the codes bit for bit against a reference that fixed the scales.
 */
tpk_status tpk_kv_quantize_pages_given_scales(const tpk_shape* shape, const void* k_pool, const void* v_pool,
                                              const int32_t* src_slots, const int32_t* dst_slots, int n_pages,
                                              const float* ks_chan, const float* ks_tok, const float* vs_chan,
                                              void* rec_pool, tpk_stream_t stream);

/*
 * Lossless 13-bit page format ("model quantization", section "A lossless tier
 * first": 13 bits per value, an 18.7 % saving, with a raw fallback when a plane
 * needs more than a 32-entry table).  A plane is one page-head's keys (or values):
 * 64 x 256 BF16 values, token-major.  A plane with at most 32 distinct exponent
 * fields is stored encoded (TPK_PACK13_PLANE_ENC bytes):
 *   u8 table[32]    the distinct exponent fields, ascending; unused entries 0  offset 0
 *   u8 sm[16384]    value i: (sign << 7) | 7-bit mantissa                     offset 32
 *   u8 lo4[8192]    table index bits 0-3: value 2j low nibble of byte j,
 *                   value 2j + 1 high nibble                                    offset 16416
 *   u8 hi1[2048]    table index bit 4 of value 8j + b in bit b of byte j        offset 24608
 * (8 + 5 bits per value), otherwise raw: the BF16 values (TPK_PACK13_PLANE_RAW
 * bytes).  A page-head record is a 16-byte header (u32 key-plane bytes, u32
 * value-plane bytes, two zero words) followed by the key plane and the value
 * plane; its size is 16 + both plane sizes, at most TPK_PACK13_RECORD_BYTES.
 */
#define TPK_PACK13_PLANE_ENC 26656
#define TPK_PACK13_PLANE_RAW 32768
#define TPK_PACK13_RECORD_BYTES 65552

/*
 * Pack n_pages BF16 pages into 13-bit records: page-head (src_slots[i], h) of
 * k_pool / v_pool -> record at pack_pool + (dst_slots[i] * H + h) *
 * TPK_PACK13_RECORD_BYTES (fixed-stride slots; the bytes of a slot past its
 * record's size are left unchanged).  src_slots, dst_slots: dev int32[n_pages];
 * pack_slots bounds dst_slots (0 = unchecked), shape->kv_slots bounds src_slots.
 * Pools 16-byte aligned.  An out-of-range slot skips that page-head and sets bit 0
 * of the device status word.  Lossless: tpk_kv_unpack13_pages restores every bit.
 */
tpk_status tpk_kv_pack13_pages(const tpk_shape* shape, const void* k_pool, const void* v_pool,
                               const int32_t* src_slots, const int32_t* dst_slots, int n_pages, void* pack_pool,
                               int64_t pack_slots, tpk_stream_t stream);

/*
 * Unpack n_pages pages of 13-bit records into BF16 pools: the record of page i,
 * KV head h starts rec_offsets[i * H + h] bytes into src (dev int64; 16-byte
 * aligned; fixed-stride slots or a compacted image alike) and is written to page
 * (dst_slots[i], h) of k_pool / v_pool.  src_bytes bounds the records (0 =
 * unchecked); shape->kv_slots bounds dst_slots.  A record whose header or extent
 * is invalid is skipped and sets bit 2 of the device status word (TPK_ERR_FORMAT
 * from tpk_get_device_status); an out-of-range slot sets bit 0.
 */
tpk_status tpk_kv_unpack13_pages(const tpk_shape* shape, const void* src, int64_t src_bytes,
                                 const int64_t* rec_offsets, const int32_t* dst_slots, int n_pages, void* k_pool,
                                 void* v_pool, tpk_stream_t stream);

/*
 * Exact-tier partial attention ("SYCL", section "A merge that joins the tiers":
 * paged decode with a log-sum-exp output).  For every KV head, the G query rows
 * attend BF16 tokens [tok_begin, tok_end) of one paged history whose token t lives
 * in slot page_table[t / 64], row t % 64.  The range is cut into num_splits
 * consecutive pieces on page boundaries (1 <= num_splits <= 4096); piece s writes
 * o_part[s] (dev float32 [num_splits][H*G][256]) and lse_part[s] (dev float32
 * [num_splits][H*G]).  A piece with no tokens writes the empty partial.
 * q: dev bf16 [H*G][256].  page_table: dev int32[ceil(tok_end / 64)].
 */
tpk_status tpk_decode_attn_exact(const tpk_shape* shape, const void* q, const void* k_pool, const void* v_pool,
                                 const int32_t* page_table, int tok_begin, int tok_end, int num_splits,
                                 float* o_part, float* lse_part, tpk_stream_t stream);

/*
 * 8-bit-tier partial attention ("SYCL", section "Attention that reads 8-bit
 * history").  As tpk_decode_attn_exact over pages [page_begin, page_end) of the
 * record pool, page p in slot page_table8[p] (dev int32[page_end]).  Keys enter
 * as q'_c = q_c * s_c folded once per page and score_t = r_t * sum_c q'_c kc_tc;
 * values accumulate on raw codes and are rescaled by u_c per page.
 */
tpk_status tpk_decode_attn_int8(const tpk_shape* shape, const void* q, const void* rec_pool,
                                const int32_t* page_table8, int page_begin, int page_end, int num_splits,
                                float* o_part, float* lse_part, tpk_stream_t stream);

/*
 * Log-sum-exp merge ("SYCL", section "A merge that joins the tiers"): fold
 * n_parts partials (dev o_parts [n_parts][rows][head_dim], lse_parts
 * [n_parts][rows]) into the accumulator (dev o_acc [rows][head_dim], lse_acc
 * [rows], read and written):
 *   lse = ln(exp(lse_acc) + sum_i exp(lse_i)),
 *   o   = exp(lse_acc - lse) o_acc + sum_i exp(lse_i - lse) o_i.
 * Partials with lse = -inf contribute nothing and their o is not read; a fresh
 * accumulator is (o = 0, lse = -inf).  The fold order is fixed (accumulator, then
 * parts in index order), so results are bit-reproducible.  head_dim must be 256.
 */
tpk_status tpk_merge_lse(int n_parts, int rows, int head_dim, const float* o_parts, const float* lse_parts,
                         float* o_acc, float* lse_acc, tpk_stream_t stream);

/*
 * Workspace bytes tpk_decode_hybrid_batched needs (partial results of the split
 * units, about 16 MiB; independent of the lengths).  The contents need no
 * initialisation.  tpk_workspace_init zero-fills a buffer (a convenience only).
 */
size_t tpk_hybrid_workspace_bytes(const tpk_shape* shape, int n_req);
tpk_status tpk_workspace_init(void* ws, size_t ws_bytes, tpk_stream_t stream);

/*
 * Multi-request hybrid decode ("SYCL", section "Exact tricks and a two-owner
 * decoder": requests in one launch, each with its own page metadata and its own
 * merge accumulator).  For each request b and KV head h: the exact partial over
 * its BF16 tokens [0, n_exact_tokens[b]) and the 8-bit partial over its pages
 * [0, n_int8_pages[b]), split across thread blocks of one decode launch, then
 * folded, in a fixed order, by a second small launch into o[b] (dev float32
 * [n_req][H*G][256]) and lse[b] (dev float32 [n_req][H*G]), which are
 * overwritten.
 *   q           dev bf16 [n_req][H*G][256]
 *   page_table  dev int32, flat; request b's exact-tier slots start at
 *               req_page_off[b] (host int32 [n_req + 1])
 *   page_table8 dev int32, flat; request b's 8-bit slots start at req_page_off8[b]
 *               (host int32 [n_req + 1])
 *   n_exact_tokens, n_int8_pages: host int32 [n_req]
 * The host arrays are read during the call (the split plan is built on the host
 * and passed by value to the kernels, so the call can be captured in a CUDA graph
 * once each device has seen one uncaptured call).
 * ws: dev workspace of at least tpk_hybrid_workspace_bytes(shape, n_req) bytes.
 * Calls sharing a workspace must not overlap on the GPU.
 */
tpk_status tpk_decode_hybrid_batched(const tpk_shape* shape, int n_req, const void* q, const void* k_pool,
                                     const void* v_pool, const void* rec_pool, const int32_t* page_table,
                                     const int32_t* req_page_off, const int32_t* n_exact_tokens,
                                     const int32_t* page_table8, const int32_t* req_page_off8,
                                     const int32_t* n_int8_pages, float* o, float* lse, void* ws, size_t ws_bytes,
                                     tpk_stream_t stream);

/*
 * The split plan tpk_decode_hybrid_batched makes, for inspection and sizing (host
 * only, no device work when resident_blocks > 0): for request b the thread blocks
 * (units) per KV head of the exact tier, splits_exact[b], and of the 8-bit tier,
 * splits_int8[b] (host int32 [n_req] each), and *n_units = H * the sum of both.
 * resident_blocks is the number of decode blocks the device holds at once (SMs x
 * blocks per SM), which sets the unit budget; 0 takes it from the current device
 * and shape->impl.  A segment gets at least one unit and at most one per page, an
 * empty request one empty exact unit; units carry about equal bytes.
 */
tpk_status tpk_hybrid_plan(const tpk_shape* shape, int n_req, const int32_t* n_exact_tokens,
                           const int32_t* n_int8_pages, int resident_blocks, int32_t* splits_exact,
                           int32_t* splits_int8, int32_t* n_units);

/*
 * Multi-request hybrid decode that allocates nothing and takes no workspace.
 * There is no counterpart in the pages this library follows: it exists for
 * callers that cannot hand the library device memory -- a plugin whose host
 * engine owns every device allocation and offers no way to ask for more, or a
 * runtime whose memory budget is fixed once serving starts.
 * Same arguments and results as tpk_decode_hybrid_batched, minus ws/ws_bytes.
 * Scratch: a file-scope device array of tpk_static_scratch_bytes() bytes
 * (16,842,752: the partials of the largest split plan, 2048 units), held by every
 * GPU that loads the library until the process exits.  A call whose plan needs
 * more fails with TPK_ERR_NOMEM.
 * The first call on a device resolves the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture.  Every call shares the one array and no state carries over between
 * calls that needs clearing, but calls that overlap on the GPU (for example on two
 * streams) race on it: serialise them.
 */
size_t tpk_static_scratch_bytes(void);
tpk_status tpk_decode_hybrid_batched_static(const tpk_shape* shape, int n_req, const void* q, const void* k_pool,
                                            const void* v_pool, const void* rec_pool, const int32_t* page_table,
                                            const int32_t* req_page_off, const int32_t* n_exact_tokens,
                                            const int32_t* page_table8, const int32_t* req_page_off8,
                                            const int32_t* n_int8_pages, float* o, float* lse,
                                            tpk_stream_t stream);

/*
 * Host-resident history staging ("ActiveKV", section on the host-authoritative KV
 * tier: pinned host memory holds every layer's history, the GPU a per-layer
 * staging working set of bounded size, filled by fenced asynchronous copies with
 * an explicit lifecycle, so a buffer is never reused while a copy or a kernel
 * still touches it).
 *
 * A stager owns one copy stream and two events per slot, created by
 * tpk_stager_create (not on the hot path); the slots are caller-owned device
 * buffers (16-byte aligned, slot_bytes each, on the device current at creation,
 * which must be current for every later call).  One host thread drives a stager.
 * Each slot cycles free -> staged -> acquired -> free:
 *   tpk_stager_stage    copies n_regions pinned host ranges (host_src[i], bytes[i])
 *                       to offsets slot_offset[i] of the next slot in round-robin
 *                       order, on the copy stream, after that slot's last release;
 *                       returns the slot index and its device address.  The host
 *                       ranges are read asynchronously: keep them valid until the
 *                       slot is acquired and the consumer has synchronised, or call
 *                       tpk_stager_sync.  Pageable sources are rejected.
 *   tpk_stager_acquire  makes `stream` wait for the slot's copies (call it right
 *                       before the work that reads the slot, so the copies of the
 *                       next layer overlap the current layer's decode).
 *   tpk_stager_release  records, on `stream`, that the work queued so far has
 *                       finished with the slot; the next staging into the slot
 *                       waits for it.
 * A call out of this order (staging into a slot that was not released, acquiring
 * a slot that is not staged, releasing one that is not acquired) returns
 * TPK_ERR_INVALID and changes nothing.  Not for use inside a stream capture.
 * tpk_stager_sync waits for every copy issued so far; tpk_stager_destroy waits for
 * them, then frees the stream and events (the slots stay the caller's).
 */
typedef struct tpk_stager tpk_stager;
tpk_status tpk_stager_create(int n_slots, void* const* slots, size_t slot_bytes, tpk_stager** out);
tpk_status tpk_stager_destroy(tpk_stager* stager);
tpk_status tpk_stager_stage(tpk_stager* stager, int n_regions, const void* const* host_src,
                            const size_t* slot_offset, const size_t* bytes, int* slot, void** slot_dev);
tpk_status tpk_stager_acquire(tpk_stager* stager, int slot, tpk_stream_t stream);
tpk_status tpk_stager_release(tpk_stager* stager, int slot, tpk_stream_t stream);
tpk_status tpk_stager_sync(tpk_stager* stager);
/*
 * Measured link behaviour ("Judge a representation by the bytes it stops
 * moving": a transfer model derived from the bus's measured behaviour): *ms =
 * the device time of the copies of the slot's latest staging, between events the
 * stager records on its copy stream right before the first and right after the
 * last of them (after the wait for the slot's release, so the copies alone).
 * Waits for those copies to finish; the slot's state is unchanged.
 */
tpk_status tpk_stager_copy_ms(tpk_stager* stager, int slot, float* ms);

/*
 * Incremental conversion and publication during decode ("ActiveKV": history
 * converted in the background and published to the decoder; "model
 * quantization": only whole pages older than the recent tokens become 8-bit).
 *
 * A tier manager follows the paged histories of n_req requests (page p of
 * request b in BF16 slot slots[p]; its record goes to the same slot of rec_pool),
 * in one layer or, with tpk_tiers_create_layers below, in several.  Each
 * tpk_tiers_step:
 *   1. publishes the pages whose conversion has finished (its event completed):
 *      they leave the exact tier and join the 8-bit tier;
 *   2. starts, on conv_stream, the conversion of every whole page that is now
 *      older than the recent_tokens newest tokens (after the work queued so far
 *      on decode_stream, which wrote those pages);
 *   3. fills `plan` with the step's tiers for tpk_decode_hybrid_batched: device
 *      page tables uploaded on decode_stream (use them on decode_stream), and host
 *      CSR offsets and counts valid until the next tpk_tiers_step.
 * A page is served exact until its conversion has finished, so a decode never
 * reads a record being written; the swap happens between steps.
 * tpk_tiers_update records request b's history after it grew: n_tokens and the
 * BF16 slots of its ceil(n_tokens / 64) pages (host array); a page converted or
 * being converted must keep its slot, and histories do not shrink.
 * Memory: dev_scratch (caller-owned, 256-byte aligned, tpk_tiers_device_bytes)
 * holds the page tables and conversion lists; two pinned host staging buffers
 * are allocated at creation and freed by tpk_tiers_destroy, which first waits
 * for the conversions in flight (tpk_tiers_sync waits without destroying).
 * One host thread drives a manager.
 */
typedef struct tpk_tiers tpk_tiers;
typedef struct {
  const int32_t* page_table;      /* dev: exact-tier slots, CSR by req_page_off */
  const int32_t* req_page_off;    /* host [n_req + 1] */
  const int32_t* n_exact_tokens;  /* host [n_req] */
  const int32_t* page_table8;     /* dev: 8-bit-tier slots, CSR by req_page_off8 */
  const int32_t* req_page_off8;   /* host [n_req + 1] */
  const int32_t* n_int8_pages;    /* host [n_req] */
  int pages_published;            /* pages that joined the 8-bit tier at this step */
  int pages_started;              /* conversions started at this step */
  int pages_converting;           /* conversions in flight after this step */
} tpk_tiers_plan;
size_t tpk_tiers_device_bytes(int n_req, int max_pages);
tpk_status tpk_tiers_create(const tpk_shape* shape, int n_req, int max_pages, int recent_tokens, const void* k_pool,
                            const void* v_pool, void* rec_pool, void* dev_scratch, size_t dev_scratch_bytes,
                            tpk_tiers** out);
tpk_status tpk_tiers_update(tpk_tiers* tiers, int b, int n_tokens, const int32_t* page_slots);
/*
 * The same manager over n_layers attention layers ("model quantization", "An
 * 8-bit page format shaped for its kernel": conversion only for pages fully
 * written in every layer, served exact until published).  The layers share the
 * requests' page tables: page p of request b lives in slot page_slots[p] of every
 * layer's pools (k_pools[l], v_pools[l]: dev BF16 pools; rec_pools[l]: dev record
 * pools; host arrays of n_layers pointers), so one plan serves every layer's
 * decode call.  A page becomes eligible once it is older than the recent window
 * and every layer has written it; its conversion runs in every layer on
 * conv_stream, and it is published -- in all layers at once -- at the first step
 * after one event recorded behind all of them.  host_rec_pools (NULL, or
 * n_layers pinned host record pools laid out like the device ones) receive a copy
 * of every converted record before that event ("ActiveKV", "The idea": host
 * memory holds the authoritative copy), so a published page's records are in the
 * host image too; the caller must not stage a page's records before it is
 * published.  tpk_tiers_create is this with one layer and no host pools.
 * tpk_tiers_update_layers records request b's history like tpk_tiers_update and
 * the tokens each layer has written so far (layer_written: host int32[n_layers],
 * each in [64 * (pages converted or being converted), n_tokens]); NULL, and
 * tpk_tiers_update, mean every layer has written all n_tokens.
 */
tpk_status tpk_tiers_create_layers(const tpk_shape* shape, int n_layers, int n_req, int max_pages, int recent_tokens,
                                   const void* const* k_pools, const void* const* v_pools, void* const* rec_pools,
                                   void* const* host_rec_pools, void* dev_scratch, size_t dev_scratch_bytes,
                                   tpk_tiers** out);
tpk_status tpk_tiers_update_layers(tpk_tiers* tiers, int b, int n_tokens, const int32_t* page_slots,
                                   const int32_t* layer_written);
tpk_status tpk_tiers_step(tpk_tiers* tiers, tpk_stream_t conv_stream, tpk_stream_t decode_stream,
                          tpk_tiers_plan* plan);
tpk_status tpk_tiers_sync(tpk_tiers* tiers);
tpk_status tpk_tiers_destroy(tpk_tiers* tiers);

/*
 * A serving step over pages whose lengths live on the device
 * -----------------------------------------------------------
 * The calls below take request lengths, page tables and token maps from device
 * memory, so a step captured once in a CUDA graph is replayed while requests grow,
 * shrink and change places: tpk_kv_tables_update turns old and new lengths into page
 * tables and slot maps, tpk_kv_rope_append rotates the new queries and keys and
 * stores keys and values into the pages (tpk_kv_norm_rope_append norms them first),
 * tpk_decode_attn_paged attends one new token per request, tpk_cross_attn_paged attends
 * any number of query tokens per request to paged states of another length (an encoder's,
 * or a prompt's own), tpk_window_attn_paged a request's last tokens to its own pages
 * through a window, tpk_decode_attn_shared one new token of requests that share prefixes;
 * tpk_kv_pages_fork, tpk_kv_pages_compact and tpk_kv_pages_copy keep pages that several
 * requests share.  They follow
 * the conventions above (ownership, pointers, streams, errors); their pools are
 * [slot][kv_heads][64][head_dim] of bfloat16 or float16, their page table is int32
 * [n_req][max_pages] (row b: the slots of request b's pages in order).  Queries, keys,
 * values, outputs, pools and workspaces are 16-byte aligned; lengths, tables, maps,
 * ranges, frequencies and lse need only be aligned to their elements, so a part of one
 * may be passed.  Others are refused.  There is no counterpart in the pages this library
 * follows.
 */
enum { TPK_BF16 = 0, TPK_F16 = 1 };
typedef struct {
  int kv_heads;      /* H in [1, 1024] */
  int group;         /* G query heads per KV head, in [1, 128]; query head j reads KV head j / G */
  int head_dim;      /* D: 64, 128 or 256 */
  int page_tokens;   /* must be 64 */
  int dtype;         /* of q, k, v and the pools: TPK_BF16 or TPK_F16 */
  float sm_scale;    /* softmax scale, finite; 0 selects 1/sqrt(head_dim) */
  int64_t kv_slots;  /* slots in each pool, > 0; kv_slots * kv_heads * 64 < 2^31 */
  int max_pages;     /* entries per page-table row (the attention calls), > 0 */
} tpk_paged_shape;

/*
 * Page tables and slot maps from request lengths.  Request b grows from len_old[b] to
 * len_new[b] tokens, shrinks (a draft taken back, or 0: finished) or stays.  With
 * have = ceil(len_old / 64) and want = ceil(len_new / 64) pages:
 *   - requests that shrink give back pages [want, have): in request order, then page
 *     order, they are pushed on the stack of free slots (free_slots[0 .. n_free));
 *   - requests that grow then take want - have slots each from the top of that stack,
 *     in request order: page have + j gets the j-th one below its predecessors'.
 * A request is refused (granted[b] = 0, its length and pages unchanged, its tokens'
 * slots -1) if a length is negative, if have or want exceeds max_pages, if its tokens
 * end past max_tokens, or if the stack holds too few slots for it: a request that
 * needs pages is granted when the pages taken by it and all before it -- refused for
 * want of slots or not -- are on the stack.
 *   len_old, len_new  dev int32 [n_req]
 *   page_table        dev int32 [n_req][max_pages], updated in place (entries past a
 *                     request's pages are left as they were)
 *   free_slots        dev int32 [free_cap], updated in place; n_free_in, n_free_out: dev
 *                     int32 [1] (a count out of [0, free_cap] is clamped; pages given
 *                     back past free_cap are dropped and set bit 0 of the device status)
 *   len_out           dev int32 [n_req]: the length each request has now
 *   granted           dev int32 [n_req]
 *   tok_off           dev int32 [n_req + 1]: where each request's new tokens begin (the
 *                     running sum of max(0, len_new - len_old), clamped to max_tokens)
 *   slot_map          dev int64 [max_tokens]: slot * 64 + row of each new token; -1 for
 *                     a refused request's tokens and past the last one
 *   positions         dev int32 [max_tokens]: its position (0 past the last)
 *   token_req         dev int32 [max_tokens]: its request (-1 past the last)
 * n_free_out may be n_free_in, len_out may be len_old or len_new: updated in place.
 * Other outputs overlap nothing.  Capturable once the device has seen one uncaptured
 * call.  n_req in [1, 4096], n_req * max_pages < 2^31;
 * max_tokens >= 0 (its three maps may be null if 0).
 */
tpk_status tpk_kv_tables_update(int n_req, int max_pages, const int32_t* len_old, const int32_t* len_new,
                                int32_t* page_table, int32_t* free_slots, int free_cap, const int32_t* n_free_in,
                                int32_t* n_free_out, int32_t* len_out, int32_t* granted, int32_t* tok_off,
                                int64_t* slot_map, int32_t* positions, int32_t* token_req, int max_tokens,
                                tpk_stream_t stream);

/*
 * Pages that several requests share.  A request's row of the page table may name pages
 * that other rows name too: answers sampled from one prompt, the beams of a search, a
 * prompt kept for later.  shares[x] counts the holders of slot x beyond the first (0 for
 * a slot with one holder, and for a free one), so that a batch without shared pages has
 * zeros, as tpk_kv_tables_update leaves them; pages held outside the batch are counted
 * in by the caller.  A request that holds shared pages is ended or cut by the call below:
 * tpk_kv_tables_update pushes the pages it gives back whoever else holds them (it may
 * grow such a request).
 *
 * Fork, end and cut, for all requests at once.  Request b becomes the first len_keep[b]
 * tokens (len_keep NULL: all) of what request source[b] was before the call: another
 * request's history, or its own (cut where len_keep[b] is less than its length, as it was
 * otherwise); with source[b] = -1 it ends.  Whole pages are shared.  A history that ends
 * inside a page will be written on there, so that page becomes the request's alone:
 *   - a request that stays as it was keeps its pages;
 *   - if nobody else holds the page after the call, the first request in order that asks
 *     for it keeps it;
 *   - every other one gets a new slot, copy_dst[b], for the rows of slot copy_src[b], which
 *     tpk_kv_pages_copy then moves.
 * First the slots that nobody holds any more are pushed on the stack of free slots, the
 * highest first; then the new slots are taken from its top, in request order.  A request
 * for whose copy no slot is left, or whose turn brings an entry of the stack that is outside
 * the pool (it is taken off all the same), keeps its whole pages only; one whose source or
 * len_keep is out of range (or more than its source has) stays as it was: both have
 * granted[b] = 0.
 *   source, len_in, len_keep  dev int32 [n_req]; len_in: the lengths before the call
 *   table_in, table_out  dev int32 [n_req][max_pages], without a common part; entries of table_out
 *                        past a request's pages are left as they were
 *   shares_in, shares_out     dev int32 [kv_slots] (may be the same)
 *   free_slots           dev int32 [free_cap], updated in place (what is not on the stack
 *                        afterwards is left as it was); n_free_in, n_free_out: dev
 *                        int32 [1] (may be the same; a count out of [0, free_cap] is
 *                        clamped; slots pushed past free_cap are dropped)
 *   len_out              dev int32 [n_req] (may be len_in); granted: dev int32 [n_req]
 *   copy_src, copy_dst   dev int32 [n_req]: -1 where nothing is copied
 * Lengths out of [0, 64 * max_pages] are clamped into it, and what is kept of such a history
 * goes by the clamped one; table entries outside the pool are left out.  Both set bit 0 of the
 * device status, and so do entries of the stack outside the pool that are taken, more releases
 * of a slot than it has holders, and dropped slots.  Outputs overlap nothing else.
 * ws: dev workspace of tpk_kv_pages_workspace_bytes(kv_slots, n_req) bytes, 16-byte aligned
 * (no initialisation); calls sharing one must not overlap on the GPU.  n_req in [1, 4096],
 * n_req * max_pages < 2^31, kv_slots + free_cap < 2^31 - 8192.  Capturable once the device has
 * seen one uncaptured call.
 */
size_t tpk_kv_pages_workspace_bytes(int64_t kv_slots, int n_req);
tpk_status tpk_kv_pages_fork(int n_req, int max_pages, int64_t kv_slots, const int32_t* source, const int32_t* len_in,
                             const int32_t* len_keep, const int32_t* table_in, int32_t* table_out,
                             const int32_t* shares_in, int32_t* shares_out, int32_t* free_slots, int free_cap,
                             const int32_t* n_free_in, int32_t* n_free_out, int32_t* len_out, int32_t* granted,
                             int32_t* copy_src, int32_t* copy_dst, void* ws, size_t ws_bytes, tpk_stream_t stream);

/*
 * Compaction: pages move from the top of the pool into free slots at its bottom, so that
 * the pool's end can be given back.  The slots not on the stack are in use.  The r-th
 * lowest free slot takes the page of the r-th highest slot in use, for as long as that is
 * higher and r < max_copies (few at a time, over several calls, or all at once).
 *   n_tokens             dev int32 [n_req]: tokens of each table row
 *   table_in, table_out  dev int32 [n_req][max_pages] (may be the same): the rows' pages
 *                        get their new slots, other entries of table_out are left alone
 *   shares_in, shares_out     dev int32 [kv_slots] (may be the same): holders go along
 *   free_in, free_out    dev int32 [free_cap] (may be the same): free_out is the stack
 *                        afterwards, the lowest slot on top; n_free_in, n_free_out: dev
 *                        int32 [1] (may be the same)
 *   new_slot             dev int32 [kv_slots]: where the page of each slot in use is now
 *                        (for holders outside the batch); -1 for the free ones
 *   copy_src, copy_dst   dev int32 [max_copies], -1 past the last; n_copies: dev int32 [1].
 *                        tpk_kv_pages_copy moves the pages: no slot is in both lists.
 * Free entries outside the pool, table entries that are on the stack or outside the pool
 * (left as they are), lengths out of range and a full stack set bit 0 of the device status.
 * Workspace, limits and capture as for tpk_kv_pages_fork; max_copies in
 * [0, 2^31 - 16384).
 */
tpk_status tpk_kv_pages_compact(int n_req, int max_pages, int64_t kv_slots, const int32_t* n_tokens,
                                const int32_t* table_in, int32_t* table_out, const int32_t* shares_in,
                                int32_t* shares_out, const int32_t* free_in, int32_t* free_out, int free_cap,
                                const int32_t* n_free_in, int32_t* n_free_out, int32_t* new_slot, int max_copies,
                                int32_t* copy_src, int32_t* copy_dst, int32_t* n_copies, void* ws, size_t ws_bytes,
                                tpk_stream_t stream);

/*
 * Copies pages within the pools of n_layers layers: slot src[i] to slot dst[i], of every
 * pool.  Pairs with a negative slot are skipped (the lists of the two calls above as they
 * are), pairs outside the pool too, setting bit 0 of the device status.  No slot may be the
 * destination of two pairs, nor a source and a destination (a pair of equal slots is
 * skipped).
 *   k_pools, v_pools     host arrays of n_layers device pools [kv_slots][kv_heads][64][head_dim]
 *   src, dst             dev int32 [n_pages]
 * Of the shape kv_heads, head_dim, dtype and kv_slots count.  n_layers in [1, 4096]; n_pages
 * in [0, 2^31 - 16384) (0 is a no-op).
 */
tpk_status tpk_kv_pages_copy(const tpk_paged_shape* shape, int n_layers, void* const* k_pools, void* const* v_pools,
                             int n_pages, const int32_t* src, const int32_t* dst, tpk_stream_t stream);

/*
 * Rotary positions with up to four axes, and the store of new keys and values into
 * their pages.  Token t's row of q (or k) is [heads][D] at q + t * q_stride elements.
 * The first rot_dim channels of each head are rotated, pair j of rot_dim / 2 by the
 * angle positions[axis_of[j]][t] * inv_freq[j]:
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 * where pair j is channels (j, j + rot_dim / 2), or (2 j, 2 j + 1) if interleaved; the
 * other channels are copied.  The angle is reduced in fixed point and rounded to float32
 * then, off by at most 2^-26 + 2^-31 turns at any 32-bit position; the products run in
 * float32 and are rounded once.
 * Rotated queries go to q_out (rows of q_out_stride elements; may be q itself with the
 * same stride), rotated keys and the values to row slot_map[t] of the pools.
 * A token with a negative slot is padding: its rows of q_out and of the pools are left
 * as they were; one with a slot past kv_slots * 64 is left out too and sets bit 0 of
 * the device status.  Tokens of one call must have distinct slots.
 *   positions  dev int32 [n_axes][n_tokens]
 *   axis_of    host uint8 [rot_dim / 2], each < n_axes; NULL: axis 0 everywhere
 *   inv_freq   dev float32 [rot_dim / 2], below 2^32 in size (others, infinities and NaN
 *              turn their pairs into NaN)
 *   slot_map   dev int64 [n_tokens]; NULL only without keys (every row is then live)
 * q and q_out may both be NULL (store only); k, v and both pools may all be NULL
 * (rotate q only).  n_tokens = 0 is a no-op; what has a row per token may then be null.
 * rot_dim is a multiple of 16, at most head_dim; 0 stores k as it is
 * (positions and inv_freq are then not read).  Strides are multiples of 8 elements, at
 * least heads * head_dim; shape->max_pages and sm_scale are not used.  Capturable once
 * the device has seen one uncaptured call.
 */
tpk_status tpk_kv_rope_append(const tpk_paged_shape* shape, int n_tokens, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* positions, int n_axes, const uint8_t* axis_of, const float* inv_freq,
                              int rot_dim, int interleaved, const int64_t* slot_map, void* q_out,
                              int64_t q_out_stride, void* k_pool, void* v_pool, tpk_stream_t stream);

/*
 * The same with a norm of each head first: query and key heads x become
 *   y_c = x_c * w_c / sqrt(sum_c x_c^2 / D + eps),  c over the head's D channels,
 * w being q_weight or k_weight, and are then rotated (or, with rot_dim 0, only stored).
 * Values are stored as they are.  Sums and products run in float32 and are rounded once;
 * values of any size are taken (the squares are scaled where float32 would not hold
 * them).  A head of zeros stays zero if eps > 0; a head with an infinity or a NaN
 * becomes what the formula gives (NaN where it is infinite over infinite).
 *   q_weight, k_weight  dev [D] of shape->dtype, 16-byte aligned; NULL: ones
 *   eps                 finite, not negative
 * The other arguments, and what is refused, as for tpk_kv_rope_append.
 */
tpk_status tpk_kv_norm_rope_append(const tpk_paged_shape* shape, int n_tokens, const void* q, int64_t q_stride,
                                   const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                   const void* q_weight, const void* k_weight, float eps, const int32_t* positions,
                                   int n_axes, const uint8_t* axis_of, const float* inv_freq, int rot_dim,
                                   int interleaved, const int64_t* slot_map, void* q_out, int64_t q_out_stride,
                                   void* k_pool, void* v_pool, tpk_stream_t stream);

/*
 * Attention of one new token per request over its pages.  Request b's query heads
 * attend tokens [tok_begin[b], n_tokens[b]) (tok_begin NULL: from 0; a sliding window
 * otherwise); token t lives in row t % 64 of slot page_table[b][t / 64].  The work is
 * split into equal page ranges over the whole device whatever the lengths, and joined
 * in a fixed order by a second small launch, so results are bit-reproducible.
 *   q          dev [n_req] rows of q_stride elements, [H*G][D]
 *   n_tokens, tok_begin: dev int32 [n_req] (values out of [0, 64 * max_pages] are
 *              clamped into it and set bit 0 of the device status)
 *   o          dev [n_req] rows of o_stride elements, [H*G][D]: of shape->dtype, or
 *              float32 if o_f32 (what tpk_merge_lse folds with other tiers' partials)
 *   lse        dev float32 [n_req][H*G]
 * A request that sees nothing gets o = 0, lse = -inf; a query row with a NaN gets NaN in
 * both.  Keys and values that are attended must be finite (an infinite value makes its
 * channel infinite or NaN).  Pool rows outside the attended range may hold anything, NaN
 * and infinities too.  A page-table entry outside the pool
 * is skipped and sets bit 0 of the device status.
 * ws: dev workspace of tpk_decode_paged_workspace_bytes(shape, n_req) bytes (no
 * initialisation; enough for fewer requests too); calls sharing one must not overlap on
 * the GPU.  n_req in [1, 4096].  Strides are multiples of 8 elements, at least H*G*D.
 * Capturable once the device has seen one uncaptured attention call of the same head_dim
 * and dtype, whatever its other arguments.
 */
size_t tpk_decode_paged_workspace_bytes(const tpk_paged_shape* shape, int n_req);
tpk_status tpk_decode_attn_paged(const tpk_paged_shape* shape, int n_req, const void* q, int64_t q_stride,
                                 const void* k_pool, const void* v_pool, const int32_t* page_table,
                                 const int32_t* n_tokens, const int32_t* tok_begin, void* o, int64_t o_stride,
                                 int o_f32, float* lse, void* ws, size_t ws_bytes, tpk_stream_t stream);

/*
 * Cross attention of ragged queries to paged states of another length.  Query tokens
 * q_off[b] .. q_off[b + 1] - 1 of request b attend its states [0, n_tokens[b]), each
 * with its own part of them if kv_range is given: query token i sees states
 * [kv_range[i][0], kv_range[i][1]) of its request (clips of a video, images before a
 * token; (0, i + 1) is a causal prompt).  Ranges are cut to [0, n_tokens[b]); an empty
 * one gives o = 0 and lse = -inf.
 *   q          dev [n_q] rows of q_stride elements, [H*G][D]
 *   q_off      dev int32 [n_req + 1], not decreasing (values are clamped into [0, n_q];
 *              rows of o and lse outside [q_off[0], q_off[n_req]) are left as they were)
 *   n_tokens   dev int32 [n_req] (clamped as above); kv_range: dev int32 [n_q][2] or NULL
 *   o          dev [n_q] rows of o_stride elements, of shape->dtype; lse: dev float32
 *              [n_q][H*G]
 * States within n_tokens[b] must be finite; pool rows past it may hold anything.  Scores
 * (sm_scale times a query times a state) past 2^22 in size in float16, 2^28 in bfloat16, whose
 * differences float32 no longer holds, may turn their row's o and lse into NaN; they never leave
 * a row finite and wrong.
 * ws: dev workspace of tpk_cross_paged_workspace_bytes(shape, n_req, n_q) bytes (no
 * initialisation), which is enough for every call of the same shape with no more requests
 * and no more query tokens; calls sharing one must not overlap on the GPU.  n_req in [1, 4096];
 * n_q >= 0 (0 is a no-op; q, kv_range, o, lse and ws may then be null).  Strides, errors
 * and capture as for tpk_decode_attn_paged.
 */
size_t tpk_cross_paged_workspace_bytes(const tpk_paged_shape* shape, int n_req, int n_q);
tpk_status tpk_cross_attn_paged(const tpk_paged_shape* shape, int n_req, int n_q, const void* q, int64_t q_stride,
                                const int32_t* q_off, const void* k_pool, const void* v_pool,
                                const int32_t* page_table, const int32_t* n_tokens, const int32_t* kv_range, void* o,
                                int64_t o_stride, float* lse, void* ws, size_t ws_bytes, tpk_stream_t stream);

/*
 * tpk_decode_attn_paged for requests that share prefixes.  Requests grp_off[g] ..
 * grp_off[g + 1] - 1 form group g: their first n_shared[g] tokens are the same (pages that
 * their table rows name together, as tpk_kv_pages_fork leaves them, and the rows of a page in
 * which the prefix ends, of which each has a copy).  The prefix is read once for the whole
 * group, from the row of its first request that has the most of it; what a request has
 * beyond it, from its own row.  Results are those of tpk_decode_attn_paged without
 * tok_begin, to rounding (where o is of the pools' type, the prefix's weights are rounded once
 * to it before the product with the values), and bit-reproducible.  The two sides are joined by their maxima
 * and sums: equal scores weigh the same on both, however far out they are.
 *   n_tokens   dev int32 [n_req], the prefix counted in; a request with fewer tokens than
 *              n_shared[g] sees those it has, one with none gets o = 0, lse = -inf
 *   grp_off    dev int32 [n_grp + 1], not decreasing (values are clamped into [0, n_req]);
 *              requests in no group share nothing
 *   n_shared   dev int32 [n_grp] (clamped as n_tokens)
 *   q, o, lse  as for tpk_decode_attn_paged
 * Pages are read as far as some request's n_tokens reach; keys and values of all tokens
 * below them must be finite, rows past them may hold anything.  NaN queries, errors, strides
 * and capture as for tpk_decode_attn_paged, scores that are too large as for
 * tpk_cross_attn_paged.
 * ws: dev workspace of tpk_decode_shared_workspace_bytes(shape, n_req, n_grp) bytes (no
 * initialisation; enough for fewer requests, and any number of groups, too); calls sharing
 * one must not overlap on the GPU.  n_req in [1, 4096], n_grp in [1, 4096].
 */
size_t tpk_decode_shared_workspace_bytes(const tpk_paged_shape* shape, int n_req, int n_grp);
tpk_status tpk_decode_attn_shared(const tpk_paged_shape* shape, int n_req, int n_grp, const void* q, int64_t q_stride,
                                  const void* k_pool, const void* v_pool, const int32_t* page_table,
                                  const int32_t* n_tokens, const int32_t* grp_off, const int32_t* n_shared, void* o,
                                  int64_t o_stride, int o_f32, float* lse, void* ws, size_t ws_bytes,
                                  tpk_stream_t stream);

/*
 * Attention through a sliding window whose first tokens stay visible, over a request's own
 * pages: one new token per request, prompts, or parts of prompts behind what is there
 * already.  Query tokens q_off[b] .. q_off[b + 1] - 1 are request b's last ones: with c of
 * them, token i of these stands at position x = n_tokens[b] - c + i and sees the tokens
 * t <= x of its request with t > x - window or t < n_sinks.  window 0: no limit (a causal
 * prompt); n_sinks 0: a plain window.  A query token in front of its request's first one
 * (c > n_tokens[b]) sees nothing: o = 0, lse = -inf.
 *   q          dev [n_q] rows of q_stride elements, [H*G][D]
 *   q_off      dev int32 [n_req + 1] as for tpk_cross_attn_paged; NULL: one query token per
 *              request (n_q = n_req)
 *   n_tokens   dev int32 [n_req], the query tokens counted in (clamped as above)
 *   o, lse     as for tpk_cross_attn_paged
 * Only pages with a token that is seen are read: the table's entries of the others may be
 * anything, so that pages behind a window may be given back.  In the pages that are read,
 * the keys and values of all tokens below n_tokens[b] must be finite; rows past it may hold
 * anything.  NaN queries, scores that are too large, errors, strides and capture as for
 * tpk_cross_attn_paged.
 * ws: dev workspace of tpk_window_paged_workspace_bytes(shape, n_req, n_q) bytes (no
 * initialisation), which is enough for every call of the same shape with no more requests
 * and no more query tokens, whatever its window; calls sharing one must not overlap on the
 * GPU.  window and n_sinks >= 0.
 */
size_t tpk_window_paged_workspace_bytes(const tpk_paged_shape* shape, int n_req, int n_q);
tpk_status tpk_window_attn_paged(const tpk_paged_shape* shape, int n_req, int n_q, int window, int n_sinks, const void* q,
                                 int64_t q_stride, const int32_t* q_off, const void* k_pool, const void* v_pool,
                                 const int32_t* page_table, const int32_t* n_tokens, void* o, int64_t o_stride,
                                 float* lse, void* ws, size_t ws_bytes, tpk_stream_t stream);

/*
 * Measurement hook: while set, every decode-kernel launch of the library (the
 * partial calls and the decode launch of the multi-request call, not its fold) is
 * preceded by a record of `before` and followed by a record of `after` on the
 * launch stream (cudaEvent_t created with timing enabled), as external records, so
 * a CUDA graph captured meanwhile records them on each replay and
 * cudaEventElapsedTime(before, after) is the decode kernel's own duration.  Both
 * null clears it.  Process-wide; set it only while no other thread launches.
 */
tpk_status tpk_set_decode_timing_events(void* before, void* after);

/*
 * Test hook for the bounded device-side waits (no counterpart in the pages: it
 * lets a test make a wait run out without faulting or hanging the GPU).  Every
 * wait of a decode or paged attention kernel on an mbarrier (for a copy to land, for a partner warp,
 * for a slot to be released) gives up after wait_limit_ns of wall time -- 0
 * restores the default of two seconds -- then sets bit 1 of the device status
 * word, lets the copies it issued land (each such wait bounded the same way) and
 * returns without writing its partial.  stall_unit >= 0 makes the tensor-core
 * decode kernel's thread block of that index (a split unit; tpk_hybrid_plan gives
 * the layout) leave its first history item unissued: no copy is made and nothing
 * arrives on that item's barrier, so the waits on it run out; the results of that
 * launch are then undefined.  In the paged attention kernels it is the block's first
 * page, or key tile.  -1 turns it off.  Process-wide, for the launches made while it
 * is set; set it only while no other thread launches.
 * Returns TPK_ERR_INVALID for stall_unit < -1 or a limit above 60 s.
 */
tpk_status tpk_set_test_wait(uint64_t wait_limit_ns, int stall_unit);

/*
 * Device status word: bit 0 = a page-table entry outside the pool was skipped,
 * bit 1 = a bounded device-side wait gave up, bit 2 = a malformed 13-bit record was
 * skipped.  Synchronises `stream`, stores the word in *flags and, if reset != 0,
 * clears it; returns TPK_ERR_TIMEOUT, TPK_ERR_BOUNDS or TPK_ERR_FORMAT (in that
 * order of precedence) when a bit is set.
 */
tpk_status tpk_get_device_status(int* flags, int reset, tpk_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* TPK_H */
