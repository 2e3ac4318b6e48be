/*
 * hdpattn.h -- C ABI of libhdpattn.so: document-masked causal attention over
 * a packed, mixed-length micro-batch, with the sequences cut into chunks of at
 * most C tokens, the causal (query chunk, key chunk) blocks computed as partial
 * (O, LSE) results, and the partials merged exactly by log-sum-exp.  One GPU
 * (sm_103a); everything runs in this library's CUDA kernels.
 *
 * Source of the method: "ByteScale: Communication-Efficient Scaling of LLM
 * Training with a 2048K Context Length on 16384 GPUs" (AI training network
 * primer research digest):
 *   section 1      capacity C: each rank holds at most C tokens;
 *   section 2      attention work grows as the square of each sequence length,
 *                  so equal-token micro-batches carry unequal FLOPs;
 *   section 3.1    a sequence longer than C spans ceil(s/C) ranks, shorter ones
 *                  are packed onto one rank by best fit (Figure 2);
 *   section 3.2    a query attends only to its own sequence; each ring step
 *                  computes one C x C block whose partial results are combined.
 *
 * Conventions for every call:
 *   - Pointers named d_* and every tensor argument are DEVICE pointers on the
 *     current CUDA device; other pointers are host pointers.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     All work is enqueued asynchronously on it; the only call that blocks the
 *     host is hdp_plan_create (one small device-to-host read of totals) and
 *     hdp_device_status (which synchronizes the stream by design).
 *   - The caller owns every buffer it passes and must keep it alive until the
 *     stream has finished the work.  A plan owns its tables.
 *   - Errors are reported only through the return code; nothing aborts and no
 *     exception crosses the ABI.  hdp_last_error_message() gives a thread-local
 *     human-readable reason for the last failing call on this thread.
 *   - Layouts: Q and O are [T][hq][d] bf16, K and V are [T][hkv][d] bf16, all
 *     row-major and contiguous; LSE is [hq][T] fp32 in natural log.  Query head
 *     h reads key/value head h / (hq / hkv).  T = total tokens, at most 2^31-1.
 */
#ifndef HDPATTN_H_
#define HDPATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  HDP_OK = 0,
  HDP_ERR_INVALID_ARGUMENT = 1, /* a documented precondition does not hold   */
  HDP_ERR_UNSUPPORTED = 2,      /* valid, but outside what the kernels cover  */
  HDP_ERR_OUT_OF_MEMORY = 3,    /* a device allocation failed                 */
  HDP_ERR_CUDA = 4,             /* a CUDA runtime/driver call failed          */
  HDP_ERR_DEVICE_TIMEOUT = 5    /* a kernel's bounded wait expired (see hdp_device_status) */
} hdp_status_t;

/* Attention modes. */
#define HDP_MODE_FUSED 0 /* every query tile runs over all its causal-prior key
                            tiles; the chunk partials are merged in registers
                            by the online softmax (exactly the LSE merge) */
#define HDP_MODE_SPLIT 1 /* each causal block (qc, kc) is written as a partial
                            (O, LSE) to the workspace, then hdp_lse_merge runs */

/* Plan creation flags. */
#define HDP_PLAN_DEFAULT 0u
#define HDP_PLAN_NO_SHARDS 1u /* skip best-fit shard packing (num_shards = 0,
                                 shard_of_chunk = NULL); for callers that only
                                 need the attention tables */
#define HDP_PLAN_NO_SPLIT 2u  /* skip the SPLIT work list (num_tiles_split = 0,
                                 tiles_split = NULL), a table for callers that
                                 schedule blocks themselves; this library's
                                 FUSED and SPLIT attention both walk the fused
                                 list and run on such a plan unchanged */

typedef struct hdp_plan_s* hdp_plan_t;

/* Read-only view of a plan.  All table pointers are device pointers owned by
 * the plan; they stay valid until hdp_plan_destroy. */
typedef struct {
  int32_t num_docs;      /* n                                                  */
  int32_t capacity;      /* C                                                  */
  int32_t num_chunks;    /* N_c = sum_i ceil(s_i / C)                          */
  int32_t num_shards;    /* shards after packing (0 with HDP_PLAN_NO_SHARDS)   */
  int64_t num_blocks;    /* N_b = sum_i n_i (n_i + 1) / 2 causal (qc, kc) blocks */
  int64_t total_tokens;  /* T                                                  */
  int32_t max_doc_len;   /* longest document                                   */
  int32_t tile;          /* query/key tile rows used by the work lists (128)   */
  const int32_t* cu_seqlens;     /* [n+1] exclusive prefix sum of lengths       */
  const int32_t* chunk_offsets;  /* [n+1] first global chunk of each document   */
  const int64_t* block_offsets;  /* [n+1] first block of each document          */
  const int32_t* chunk_table;    /* [N_c][4] {doc, index in doc, first token, length} */
  const int32_t* block_table;    /* [N_b][2] {q chunk, kv chunk}, ordered by doc,
                                    then q chunk, then kv chunk ascending      */
  const int64_t* chunk_pairs;    /* [N_c] causal (query, key) pairs per chunk  */
  const int32_t* shard_of_chunk; /* [N_c] shard of each chunk (NULL if skipped) */
  /* Query-tile work lists, heaviest first (weight descending, then
   * enumeration order).  Rows of 8 int32: {q_row0, q_rows, kv_row0, kv_len,
   * block (-1 in the fused list), row offset of the tile inside its query
   * chunk (inside its document in the fused list), weight = key tiles,
   * document length (fused list; 0 in the split list)}.  Fully masked
   * (cross-document or future) tiles never appear.  In the fused list the
   * rows of query tile j of a document also describe its key tile j (same
   * rows), which the backward pass walks.  Both attention modes walk the
   * fused list; the split list is a table for callers that schedule one
   * causal block at a time. */
  const int32_t* tiles_fused;    /* [num_tiles_fused][8] one per document query tile */
  int64_t num_tiles_fused;
  const int32_t* tiles_split;    /* [num_tiles_split][8] one per block query tile
                                    (NULL unless C is a multiple of `tile`)   */
  int64_t num_tiles_split;
} hdp_plan_view_t;

/*
 * Sharding plan (section 3.1, Figure 2): chunk every document into
 * ceil(s/C) chunks of at most C tokens, enumerate the causal blocks
 * (qc, kc), kc <= qc, of each document, count the causal pairs of each chunk,
 * pack the chunks into shards (every full C-token chunk gets its own shard in
 * chunk order; shorter pieces -- short documents and tails -- are packed by
 * best-fit decreasing: length descending, document ascending, each into the
 * open piece shard with the least remaining capacity that fits, lowest id on
 * ties, else a new shard), and build the query-tile work lists.
 *   d_lengths  [num_docs] int32 device array, every entry >= 1.
 *   num_docs   >= 1.      capacity >= 1.
 *   flags      HDP_PLAN_DEFAULT, or HDP_PLAN_NO_SHARDS and / or
 *              HDP_PLAN_NO_SPLIT OR-ed together.
 *   out        receives the plan (NULL on failure).
 * Blocks the host once, to read the totals and the shard count back (best fit
 * runs on the device before that read-back).  Fails with INVALID_ARGUMENT for a
 * length < 1 or T >= 2^31, UNSUPPORTED when more than 65,536 sub-capacity
 * pieces need best-fit packing (use HDP_PLAN_NO_SHARDS), OUT_OF_MEMORY if the
 * tables cannot be allocated.  Tables are allocated stream-ordered on
 * `stream`.
 */
hdp_status_t hdp_plan_create(const int32_t* d_lengths, int32_t num_docs, int32_t capacity, void* stream,
                             hdp_plan_t* out);
hdp_status_t hdp_plan_create_ex(const int32_t* d_lengths, int32_t num_docs, int32_t capacity, uint32_t flags,
                                void* stream, hdp_plan_t* out);
hdp_status_t hdp_plan_view(hdp_plan_t plan, hdp_plan_view_t* view);
/* Frees the plan's tables, stream-ordered on the stream the plan was created
 * on; work on other streams that uses the plan must be ordered before it. */
hdp_status_t hdp_plan_destroy(hdp_plan_t plan);

/*
 * Workspace bytes hdp_attention_fwd needs for (plan, hq, d, mode).  FUSED needs
 * none (0).  SPLIT needs the partials: N_b * C * hq * (d + 1) * 4 bytes, laid
 * out as o_part [N_b][C][hq][d] fp32 followed by lse_part [N_b][hq][C] fp32
 * (256-byte aligned), the format hdp_lse_merge reads.
 */
hdp_status_t hdp_attention_workspace_bytes(hdp_plan_t plan, int32_t hq, int32_t d, int32_t mode, size_t* bytes);

/*
 * Document-masked causal attention forward (section 3.2): for every document,
 * query head h and doc-local query p,
 *   S_j = scale * q_p . k_j for doc-local keys j <= p,
 *   lse = ln sum_j exp(S_j),  o = sum_j exp(S_j - lse) v_j,
 * with query tiles scheduled heaviest first and fully masked tiles skipped.
 *   q [T][hq][d], k/v [T][hkv][d] bf16; o [T][hq][d] bf16 (round to nearest
 *   even); lse [hq][T] fp32 (natural log).
 *   hq % hkv == 0; d == 64 or 128 (else UNSUPPORTED); scale > 0.
 *   FUSED: o and lse are final.  SPLIT: needs capacity % 128 == 0 and a
 *   workspace of hdp_attention_workspace_bytes; writes the partials there,
 *   then merges them into o and lse with hdp_lse_merge on the same stream.
 *   Each partial covers exactly its block's C keys: the kernel walks the
 *   fused list and writes a partial at every chunk end of a query tile's
 *   key range.
 *   When one kv head's K and V rows of the longest document exceed the
 *   device's L2, the CTAs of a launch pace each other along the key range so
 *   that they share K/V tiles in L2.  Their positions go through one static
 *   device table (its address cached per device, like the scratch of
 *   hdp_attention_fwd_split_noalloc); concurrent launches share it, which can
 *   only weaken the pacing (every hold is bounded) and never changes the
 *   results.
 *   q, k, v, o must be 16-byte aligned.
 *   Sums of products are cut off, not rounded, in fp32: outputs of rows that see n
 *   keys of like weight are too small by about n 2^-27.5 of themselves (0.6 % at 1M).
 * Device-side wait timeouts are reported by hdp_device_status.
 */
hdp_status_t hdp_attention_fwd(hdp_plan_t plan, const void* q, const void* k, const void* v, int32_t hq,
                               int32_t hkv, int32_t d, float scale, int32_t mode, void* workspace,
                               size_t workspace_bytes, void* o, float* lse, void* stream);

/*
 * SPLIT-mode attention that allocates nothing.  The paper has no counterpart;
 * this entry exists for callers that cannot allocate device memory at the time
 * they run attention: serving processes that reserve all device memory at
 * start-up and forbid allocation on the request path, host programs whose own
 * allocator owns the device memory, and callers that must avoid the
 * device-wide synchronisation cudaMalloc/cudaFree can imply.
 * Same arguments and results as hdp_attention_fwd with mode HDP_MODE_SPLIT,
 * but the partials live in a fixed 64 MiB scratch array inside the library
 * (every GPU that loads the library holds it until the process exits).
 *   - Plans whose SPLIT workspace (hdp_attention_workspace_bytes) exceeds
 *     64 MiB are rejected with HDP_ERR_INVALID_ARGUMENT and a message.
 *   - No cudaMalloc, cudaFree or other allocating call is made.  The first
 *     call on a device resolves the scratch array's device address (once per
 *     device, with that device current) and caches it.  A cudaDeviceReset,
 *     or anything else that destroys the device's primary context,
 *     invalidates the cached address (and those of the device error word and
 *     the attention pacing table): do not call the library on that device
 *     after such a reset in the same process.
 *   - Every call shares the one scratch array, which keeps the last call's
 *     contents; every partial a call reads is written by that call first, so
 *     nothing needs to start at zero.  Calls that overlap on the GPU (other
 *     streams, other threads) race on the array and must be serialised by the
 *     caller.
 */
hdp_status_t hdp_attention_fwd_split_noalloc(hdp_plan_t plan, const void* q, const void* k, const void* v,
                                             int32_t hq, int32_t hkv, int32_t d, float scale, void* o, float* lse,
                                             void* stream);

/*
 * Backward pass of the same attention (the training step of section 5 times
 * forward and backward together; each document's gradient is independent,
 * section 3.2).  With P = exp(scale Q K^T - lse) over the causal keys of each
 * query's own document and D = rowsum(dout * o):
 *   dv = P^T dout,  dS = P * (dout V^T - D),  dk = scale dS^T Q,  dq = scale dS K
 * summed over the query heads of each GQA group for dk and dv.
 *   q, o, dout, dq: [T][hq][d] bf16;  k, v, dk, dv: [T][hkv][d] bf16;
 *   lse: [hq][T] fp32, natural log, as written by hdp_attention_fwd for this
 *   plan (FUSED or SPLIT) and `o` its output.
 * workspace: device, 256-byte aligned, at least
 * hdp_attention_bwd_workspace_bytes (D in fp32).  Deterministic: no atomics;
 * dq, dk and dv each accumulate in one CTA in a fixed order.
 * d == 64 or 128 (UNSUPPORTED otherwise); tensor pointers 16-byte aligned.
 * Every output row is written.
 */
hdp_status_t hdp_attention_bwd_workspace_bytes(hdp_plan_t plan, int32_t hq, int32_t d, size_t* bytes);
hdp_status_t hdp_attention_bwd(hdp_plan_t plan, const void* q, const void* k, const void* v, const void* o,
                               const float* lse, const void* dout, int32_t hq, int32_t hkv, int32_t d, float scale,
                               void* workspace, size_t workspace_bytes, void* dq, void* dk, void* dv, void* stream);

/*
 * Exact log-sum-exp merge of the causal blocks of every query chunk
 * (section 3.2: the partial results of the ring steps are combined):
 *   M = max_k lse_k, lse = M + ln sum_k exp(lse_k - M), o = sum_k exp(lse_k - lse) o_k
 * over the blocks (qc, kc), kc = 0..qc, of the chunk.
 *   o_part [N_b][C][hq][d] fp32, lse_part [N_b][hq][C] fp32 (the SPLIT
 *   workspace layout); o [T][hq][d] bf16, lse [hq][T] fp32.  d == 64 or 128.
 *   The plan's capacity must be a multiple of 128 (as for SPLIT attention):
 *   INVALID_ARGUMENT otherwise.
 */
hdp_status_t hdp_lse_merge(hdp_plan_t plan, const float* o_part, const float* lse_part, int32_t hq, int32_t d,
                           void* o, float* lse, void* stream);

/*
 * The same merge on plain arrays: m partials of `rows` rows of d values.
 *   o_parts [m][rows][d] fp32, lse_parts [m][rows] fp32 -> o [rows][d] bf16,
 *   lse [rows] fp32.  A partial with lse = -inf contributes nothing; a row whose
 *   partials are all -inf gets lse = -inf and o = 0.  m >= 1, d % 4 == 0,
 *   d <= 256.
 */
hdp_status_t hdp_lse_merge_rows(int32_t m, int64_t rows, int32_t d, const float* o_parts, const float* lse_parts,
                                void* o, float* lse, void* stream);

/*
 * Useful causal-attention FLOPs per shard (section 2: micro-batches of equal
 * tokens differ in FLOPs): d_out[s] = sum over the shard's chunks of
 * 4 * d * hq * chunk_pairs, exact in int64.  d_out [num_shards] int64 device.
 * INVALID_ARGUMENT if the plan was created with HDP_PLAN_NO_SHARDS.
 */
hdp_status_t hdp_flops_per_shard(hdp_plan_t plan, int32_t d, int32_t hq, int64_t* d_out, void* stream);

/* ====================================================================== */
/* 8-bit key/value cache: writing it, reading it back, attention over it for
 * the newest tokens of each sequence, a cheap score that chooses blocks of it
 * for each query, and attention over the chosen blocks.  With it a packed
 * prompt that went through hdp_attention_fwd is continued token by token.
 *
 * A cache is a pool of pages of HDP_CACHE_BLOCK tokens, shared by any number
 * of sequences; a page table says which page holds block b (tokens 64 b ..
 * 64 b + 63) of sequence i.  The caller owns every buffer, hands out pages and
 * advances the lengths; nothing is kept inside the library between calls, all
 * calls are asynchronous, none blocks the host, allocates or needs a
 * workspace in a given state, and all of them may be captured into a CUDA
 * graph and replayed while the caller changes the lengths, tables and inputs
 * in place.
 *
 * Codes.  Each (page, kv head) has two scales, one for K and one for V; a
 * value is code * scale.  A scale is a power of two: the smallest 2^e,
 * e >= -126, with |x| <= M 2^e for every row ever written to the block since
 * its first one (M = 448 for e4m3, 127 for int8).  Division by it, code *
 * scale (in bf16 too, see hdp_cache_read) and a change of scale are exact but
 * for one rounding of the code to the nearest (ties to even).  When a row needs a larger scale,
 * the block's codes are rounded to the new one; over any number of such
 * changes an int8 value is off by less than one step and an e4m3 value by at
 * most half a step plus one subnormal step (2^-9 scale).  A row with an
 * infinity or NaN makes the scale NaN: the block then reads as NaN until its
 * first row is written again.
 *
 * Bounds.  For each (page, kv head) the channel-wise minimum and maximum of
 * the K rows ever written, rounded outwards to whole multiples of the K scale
 * (int8) or of four K scales (e4m3): a function of the rows alone.
 */
#define HDP_CACHE_BLOCK 64
#define HDP_CACHE_E4M3 0
#define HDP_CACHE_INT8 1

typedef struct {
  void* k;               /* [num_pages][hkv][64][d] codes, 16-byte aligned    */
  void* v;               /* [num_pages][hkv][d][64] codes, 16-byte aligned:
                            token t = 16 j + 8 h + 2 c + e of a block stands
                            at byte 16 c + 4 j + 2 h + e                       */
  float* scales;         /* [num_pages][hkv][2] {K, V}, 8-byte aligned         */
  int8_t* bounds;        /* [num_pages][hkv][2][d] {min, max}, 16-byte aligned */
  int32_t num_pages;     /* >= 1                                               */
  int32_t hkv;           /* >= 1                                               */
  int32_t d;             /* 64 or 128                                          */
  int32_t format;        /* HDP_CACHE_E4M3 or HDP_CACHE_INT8                   */
  const int32_t* page_table; /* [num_seqs][max_pages] page of each block       */
  const int32_t* lens;   /* [num_seqs] tokens of each sequence, the rows of the
                            call included                                      */
  int32_t num_seqs;      /* >= 1                                               */
  int32_t max_pages;     /* columns of page_table, >= 1                        */
} hdp_cache_t;

/*
 * Common to the calls below.  The rows of a call are the newest tokens of each
 * sequence, packed: cu [num_seqs + 1] (device int32, cu[0] = 0, ascending)
 * gives sequence i the rows cu[i] .. cu[i+1] - 1, and row r of it is the token
 * at position lens[i] - (cu[i+1] - cu[i]) + r.  cu NULL means one row for each
 * sequence; `rows` must then equal num_seqs.  `rows` is the row count of the
 * row tensors (0 .. 2^31-1); rows from cu[num_seqs] on belong to no sequence:
 * they are not read, and their outputs are left as they were.  A row at a
 * negative position (more rows than tokens) is not written, reads as zeros,
 * attends to nothing and selects nothing.
 * A length outside [0, 64 max_pages] is taken as the nearest bound, and a page
 * outside [0, num_pages) is never touched (its tokens are not written, read
 * as zeros, and are masked in the attention); both are reported by the next
 * hdp_device_status as INVALID_ARGUMENT.  Table entries beyond a sequence's
 * last block may hold anything.
 * Host-side errors: INVALID_ARGUMENT for NULL pointers, sizes, alignment and
 * workspaces; UNSUPPORTED for a d other than 64 and 128.
 */

/*
 * Writes K and V rows (bf16 [rows][hkv][d], 16-byte aligned) into the cache.
 * A block's first row starts the block anew: its codes, scales and bounds do
 * not depend on what the page held before (other rows get zero codes).  Rows
 * appended behind the first keep the codes that are there, at a larger scale
 * if the new rows need one.  Positions may be written again (a rejected draft
 * is overwritten by appending with a smaller length).  A page that the call
 * writes must belong to one sequence only; complete pages may be shared.
 */
hdp_status_t hdp_cache_append(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* k, const void* v,
                              void* stream);

/* Reads the rows back: k, v [rows][hkv][d] bf16: exactly code * scale, but for
 * e4m3 codes at scales of 2^-126 and 2^-125, whose smallest products are below
 * bf16's smallest number and are rounded to it. */
hdp_status_t hdp_cache_read(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, void* k, void* v, void* stream);

/*
 * Attention of the rows over the cache: for row r of sequence i at position p
 * and query head h (kv head h / (hq / hkv)),
 *   S_j = scale * q . k_j over cached tokens j <= p,
 *   lse = ln sum_j exp(S_j),  o = sum_j exp(S_j - lse) v_j,
 * and o = 0, lse = -inf where no token is left; o and lse are NaN for a query row
 * with an infinity or NaN that has a token left.  Inputs are the dequantised
 * codes; sums and the softmax's statistics are fp32, and a weight is rounded to 11
 * bits where it multiplies V (it is off by 2^-11 of itself at most, and o by 2^-11
 * of the sum of weight times |v|).  That holds for q, K and V
 * over all of bf16's range, scores up to 2^127 in magnitude, and weights down to 2^-126
 * of a row's largest, where weight times V scale is at least 2^-100 of the row's
 * largest such product.  (What is smaller shows in channels in which the keys above
 * it have zeros.)  Elements of a query row below 2^-31 of its largest keep fewer
 * bits (they are rounded to multiples of 2^-38 of it).
 *   q, o [rows][hq][d] bf16, 16-byte aligned; lse [hq][rows] fp32; hq % hkv == 0.
 *   blocks NULL (count 0): every block.  Else device int32 [rows][hkv][count],
 *   count >= 1: for each row and kv head the blocks to attend to, strictly
 *   ascending.  An entry that is negative, beyond the row's position or not
 *   above the entry directly before it is skipped (hdp_cache_select pads with
 *   -1).  Nothing else is checked: a block that stands twice in a list that does
 *   not ascend may count twice.
 *   workspace: device, 256-byte aligned, at least
 *   hdp_cache_attention_workspace_bytes (which depends on the device's SM
 *   count and d only: 122 MB for d = 128 on 152 SMs, 62 MB for d = 64); calls
 *   that may overlap need one each.
 * Deterministic: the order of all sums depends only on the shapes and lengths.
 * Made for a few rows per sequence (16 rows times heads of a group share one
 * pass over the cache); more rows are correct and read the cache again.
 */
hdp_status_t hdp_cache_attention_workspace_bytes(const hdp_cache_t* cache, int32_t hq, size_t* bytes);
hdp_status_t hdp_cache_attention(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* q, int32_t hq,
                                 float scale, const int32_t* blocks, int32_t count, void* workspace,
                                 size_t workspace_bytes, void* o, float* lse, void* stream);

/*
 * Chooses `count` blocks for each row and kv head by an upper bound of its
 * scores.  The query rows of the head's group are rounded to whole numbers c
 * with one power of two for the group (largest magnitude at most 127); with
 * lo, hi the bounds of a block and s its K scale,
 *   U = sum over heads and channels of max(c, 0) hi + min(c, 0) lo   (integer),
 *   score = fp32(U) * s.
 * Of the blocks 0 .. p / 64 of a row at position p, the first keep_first and
 * the last keep_last are always chosen, then those with the highest scores,
 * ties to the lower block; a block whose scale is NaN counts as highest, one
 * whose page is invalid as lowest.
 * Whole-number sums make the choice independent of any order of summation.
 * (An infinity or NaN in q counts as 0 here; the attention returns NaN.)
 *   q [rows][hq][d] bf16, 16-byte aligned, hq / hkv <= 128;
 *   blocks [rows][hkv][count] int32 out: ascending, -1 behind the last;
 *   count >= 1, keep_first >= 0, keep_last >= 0, keep_first + keep_last <= count;
 *   workspace: device, 256-byte aligned, hdp_cache_select_workspace_bytes
 *   (rows * hkv * max_pages scores of 4 bytes, also where they are not used).
 */
hdp_status_t hdp_cache_select_workspace_bytes(const hdp_cache_t* cache, int64_t rows, size_t* bytes);
hdp_status_t hdp_cache_select(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* q, int32_t hq,
                              int32_t count, int32_t keep_first, int32_t keep_last, void* workspace,
                              size_t workspace_bytes, int32_t* blocks, void* stream);

/* ====================================================================== */
/* 4-bit key/value cache: half the bytes of the 8-bit one, with finer scales and
 * the same pages, page tables, lengths, rows and rules ("Common to the calls
 * below" above holds here too, with workspaces and streams).  A row's codes
 * depend on that row alone, so rows may be written in any order and pieces, and
 * written again, and every bit of the cache that they decide is the same.
 *
 * Codes are e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 for the low three bits, the fourth
 * is the sign; two in a byte, the first in its low half.  A value is code *
 * scale.  A scale is a power of two, held in a byte as its exponent plus 127
 * (255: NaN): the smallest 2^e, e >= -126, with |x| <= 6 2^e over the 32 channels
 * of K, or over the d channels of V, that share it.  x / scale is exact and is
 * rounded to the nearest code (ties to the even one); half a step of it is at most
 * scale.  (Values beyond 3 * 2^126 are taken as that: the next code is past bf16's
 * end.)  Channels that share a scale with an infinity or NaN read as NaN.  Byte 0 is
 * never written; what is read through it is unspecified, but below 2^-124.
 */
typedef struct {
  void* k;               /* [num_pages][hkv][64][d/2], 16-byte aligned: channel
                            32 g + 8 c + 2 b + e of a token stands in byte
                            (d/8) c + 4 g + b of its row, half e                */
  void* v;               /* [num_pages][hkv][d/16][512], 16-byte aligned: channel
                            16 i + 8 h + r of token 16 s + 8 p + 2 c + e stands in
                            byte 64 r + 16 c + 8 h + 2 s + p of row i, half e   */
  uint8_t* scales;       /* [num_pages][hkv][d/32 + 1][64], 16-byte aligned: row g
                            of channels 32 g .. 32 g + 31 of K, the last row of V,
                            token 8 j + r at place 8 r + j                      */
  int32_t num_pages;     /* >= 1                                               */
  int32_t hkv;           /* >= 1                                               */
  int32_t d;             /* 64 or 128                                          */
  int32_t num_seqs;      /* >= 1                                               */
  const int32_t* page_table; /* [num_seqs][max_pages] page of each block       */
  const int32_t* lens;   /* [num_seqs] tokens of each sequence, the rows of the
                            call included                                      */
  int32_t max_pages;     /* columns of page_table, >= 1                        */
} hdp_fourbit_cache_t;

/* Writes K and V rows (bf16 [rows][hkv][d], 16-byte aligned) into the cache.
 * Nothing but their codes and scales is changed.  A page that the call writes must
 * belong to one sequence only; complete pages may be shared. */
hdp_status_t hdp_fourbit_append(const hdp_fourbit_cache_t* cache, const int32_t* cu, int64_t rows, const void* k,
                                const void* v, void* stream);

/* Reads the rows back: k, v [rows][hkv][d] bf16, exactly code * scale. */
hdp_status_t hdp_fourbit_read(const hdp_fourbit_cache_t* cache, const int32_t* cu, int64_t rows, void* k, void* v,
                              void* stream);

/* hdp_cache_attention over this cache: the same formulas, arguments and promises,
 * over all blocks (there are no lists), but that weights count down to 2^-100 of a
 * row's largest; that small ones may together lose 2^-11 of a channel's sum of weight
 * times |v| besides what each loses to rounding; and that where a row's score passes
 * fp32's end before it is multiplied by `scale`, K scales below 2^-94 may count as 0 in
 * the 64 keys of its block.  A call takes longer where the scores of a head deviate by
 * more than a nat or so: up to 1.8 times as long at 1.7 nats, 5 times at 3.4.
 * workspace: device, 256-byte aligned, at least
 * hdp_fourbit_attention_workspace_bytes, which depends on the device's SM count and
 * d only (152 SMs: 12.7 MB for d = 128, 6.4 MB for d = 64); calls that may overlap
 * need one each. */
hdp_status_t hdp_fourbit_attention_workspace_bytes(const hdp_fourbit_cache_t* cache, int32_t hq, size_t* bytes);
hdp_status_t hdp_fourbit_attention(const hdp_fourbit_cache_t* cache, const int32_t* cu, int64_t rows, const void* q,
                                   int32_t hq, float scale, void* workspace, size_t workspace_bytes, void* o, float* lse,
                                   void* stream);

/* ====================================================================== */
/* Block tables and slot maps from the requests' lengths, for either cache.
 *
 * hdp_cache_assign brings the pages that the sequences hold in line with their
 * lengths.  The free pages of a pool are a stack: free_pages [num_pages], of which
 * the first free_count[0] are free, the last of them on top.  Sequence i holds the
 * pages of its blocks 0 .. held[i] - 1, page_table [num_seqs][max_pages] says
 * which, and it needs ceil(lens[i] / 64).
 *   1. Pages beyond that go back on the stack: the last sequence's first, and of a
 *      sequence the last block's first.
 *   2. Then each sequence, in order, takes a page from the top for every block
 *      that it lacks, in order.  A sequence whose blocks are not all there, and
 *      every later one that lacks any, takes none and keeps its held[i]; the next
 *      hdp_device_status then reports OUT_OF_MEMORY, unless something else has to be
 *      reported: one call reports one failure.
 * free_pages, free_count, held and page_table are updated in place; taking pages
 * and giving them back leaves the stack as it was.  Entries of page_table beyond
 * held[i] are left as they are.  Lengths, held and free_count outside their ranges
 * are taken as the nearest bound and reported as INVALID_ARGUMENT.  All pointers
 * are device pointers; calls on one pool must not overlap.  A page belongs to one
 * sequence: pages that sequences share are not for this call to give back.
 * num_seqs at most 2^24.
 */
hdp_status_t hdp_cache_assign(int32_t* free_pages, int32_t* free_count, int32_t num_pages, int32_t* page_table,
                              int32_t* held, const int32_t* lens, int32_t num_seqs, int32_t max_pages, void* stream);

/*
 * Where the rows of a call lie (rows, cu and lens as in the cache calls):
 * sequence [rows] int32, position [rows] int32 and slot [rows] int64 = page * 64 +
 * position % 64; each may be NULL.  Rows of no sequence get -1 in all three, rows
 * at a negative position and rows on a page outside [0, num_pages) get slot -1
 * (the latter is reported like a bad page of a cache call).  page_table NULL: no
 * slots, slot must be NULL, max_pages and num_pages are ignored and lengths are
 * only bounded below, by 0: with lens the lengths of packed documents and cu their
 * prefix sums, position is each token's place in its document.
 */
hdp_status_t hdp_cache_rows(const int32_t* page_table, const int32_t* lens, const int32_t* cu, int32_t num_seqs,
                            int32_t max_pages, int32_t num_pages, int64_t rows, int32_t* sequence, int32_t* position,
                            int64_t* slot, void* stream);

/* ====================================================================== */
/* Rotary positions.  Pair i (0 .. rot/2 - 1) of a head's channels, (a, b) =
 * channels (i, i + rot/2), or with HDP_ROTARY_NEIGHBOURS (2 i, 2 i + 1), becomes
 *   (factor (a cos x - b sin x), factor (b cos x + a sin x)),  x = position * freqs[i],
 * channels from rot on are copied.  With HDP_ROTARY_BACKWARD x is negated: the
 * gradient of the rows before the turn from that of the rows behind it.
 *   q, k: either may be NULL.  Rows [rows][heads][d] of `type`, channels
 *   contiguous, other strides in elements; out may be in (with the same strides),
 *   else the two must not overlap, and neither out may overlap the other's rows or
 *   itself: such calls are refused (so are rows with different strides that lie
 *   between each other).  Any alignment; 16-byte steps where the addresses, strides
 *   and rot allow them (slower, but the same results, where rot or they do not).
 *   position [rows] int32; a row at a negative one is not read, its output is left
 *   as it was.  freqs [rot/2] double, radians, finite (device; scaling for long
 *   contexts is in them and in factor).  2 <= rot <= d <= 256, rot even; factor > 0.
 * The angle's fraction of a turn is right to 2^-31 over all positions and
 * frequencies below 2^53 in magnitude (beyond them nothing is promised) and, as a
 * fraction of half a turn, rounded to fp32.  Products and sums are fp32, rounded once
 * to `type`.
 */
#define HDP_TYPE_BF16 0
#define HDP_TYPE_FP16 1
#define HDP_TYPE_FP32 2
#define HDP_ROTARY_NEIGHBOURS 1
#define HDP_ROTARY_BACKWARD 2
typedef struct {
  const void* in;
  void* out;
  int64_t in_row_stride, in_head_stride, out_row_stride, out_head_stride;
  int32_t heads; /* 0 .. 2^20 */
} hdp_rotary_rows_t;
hdp_status_t hdp_rotary(const hdp_rotary_rows_t* q, const hdp_rotary_rows_t* k, int64_t rows, int32_t d, int32_t type,
                        const int32_t* position, const double* freqs, int32_t rot, int32_t flags, float factor,
                        void* stream);

/*
 * Synchronizes `stream` and reports (then clears) a device-side failure
 * recorded by an earlier kernel of this library on the current device:
 * HDP_ERR_DEVICE_TIMEOUT when a bounded wait expired, INVALID_ARGUMENT when a
 * cache call met a length or page outside its tables, OUT_OF_MEMORY when
 * hdp_cache_assign ran out of free pages, HDP_ERR_CUDA when the stream reports a
 * CUDA error, else HDP_OK.
 */
hdp_status_t hdp_device_status(void* stream);

const char* hdp_status_string(hdp_status_t status);
const char* hdp_last_error_message(void);

/* Number of CUDA kernels this library has enqueued in this process (all
 * devices, all threads).  Diagnostic counter; never reset. */
uint64_t hdp_kernel_launch_count(void);

/* Number of times this library has blocked the host on a stream in this
 * process: hdp_plan_create's one read-back and hdp_device_status.  Diagnostic
 * counter; never reset. */
uint64_t hdp_host_sync_count(void);

/*
 * Budget of the bounded waits of the attention forward and backward kernels,
 * in SM clocks, for the launches this process makes after the call (all
 * devices, all threads).
 * clocks <= 0 restores the default of 2e9 clocks (about one second at
 * 2 GHz); no legitimate wait lasts more than a few microseconds.  A budget of
 * a few clocks makes the first wait that is not already satisfied expire: the
 * kernel then records the expiry, stops every role, waits (on its own,
 * unchanged budget) for the copies and tensor-core work it has in flight,
 * frees its tensor memory and returns, and hdp_device_status reports
 * HDP_ERR_DEVICE_TIMEOUT.  This is how the timeout path is tested without a
 * fault; production code leaves the default.  Always returns HDP_OK.
 */
hdp_status_t hdp_set_wait_budget(int64_t clocks);

/* ====================================================================== */
/* Cost models (host arithmetic only: no device, no stream, no allocation).
 * "ByteScale: ..." research digest, section 3.2 (ring timing model and its
 * table of worked cases) and section 3.3 (cost models T(s), Act(s) and
 * Eq. 3).  Times and bandwidths are in any consistent units. */

/*
 * Per-step compute of a ring of N ranks holding C tokens each (section 3.2):
 *   t_c = t_blk * sum_i (s_i / (N C))^2
 * where every sequence of the pack is cut into N slices and a query attends
 * only to its own sequence; t_blk is the time of one full C x C block.
 * lengths: host int32[n], n >= 1, every s_i >= 1, sum s_i <= N * C.
 * INVALID_ARGUMENT otherwise (or t_blk < 0, or a null pointer).
 */
hdp_status_t hdp_ring_step_compute(const int32_t* lengths, int32_t n, int32_t num_ranks, int32_t capacity,
                                   double t_blk, double* t_c);

/*
 * Attention time of that ring (section 3.2): each step overlaps the transfer
 * of the next K/V slice (t_x) with the compute on the current one (t_c):
 *   T_attn = (N - 1) * max(t_c, t_x) + t_c.
 * num_ranks >= 1, t_c >= 0, t_x >= 0.
 */
hdp_status_t hdp_ring_attention_time(int32_t num_ranks, double t_c, double t_x, double* t_attn);

/* Profiled cost models of section 3.3, T(s) = alpha1 s^2 + beta1 s + gamma
 * (time of one layer on a sequence of s tokens) and
 * Act(s) = alpha2 s + beta2 (activation bytes of one layer), with the
 * device-to-host and host-to-device copy bandwidths (bytes per time unit)
 * and l layers per rank. */
typedef struct {
  double alpha1, beta1, gamma;
  double alpha2, beta2;
  double bw_d2h, bw_h2d;
  int32_t layers; /* l >= 3 */
} hdp_offload_model_t;

/*
 * Selective offloading, Eq. 3 (section 3.3): the rank count of a sequence of
 * s tokens when a fraction r of the activations of l - 2 of its l layers is
 * kept in host memory,
 *   D(s) = ceil((2 Act(s) + (1 - r)(l - 2) Act(s)) / (l Act(C))),
 * subject to the copy hiding behind compute, T(s) >= r Act(s) / min(B_d2h, B_h2d),
 * and to 1 >= r >= min(1, l Act(C) / ((l - 2) Act(s))).  D does not grow with r,
 * so the rank count is smallest at the largest admissible ratio:
 *   r = min(1, T(s) min(B_d2h, B_h2d) / Act(s)) when that is at least the lower
 *   bound, else r = 0 (no offloading, D = ceil(Act(s) / Act(C))).
 * Requires s >= 1, capacity >= 1, layers >= 3, Act(C) > 0, Act(s) > 0,
 * bandwidths >= 0.  Outputs the chosen ratio and rank count.
 */
hdp_status_t hdp_offload_ranks(const hdp_offload_model_t* model, int64_t s, int64_t capacity, double* r,
                               int64_t* ranks);

/*
 * Least-squares fit of a profiled cost model (section 3.3): the polynomial of
 * the given degree (1: Act(s) = c1 s + c0; 2: T(s) = c2 s^2 + c1 s + c0)
 * minimising sum_i w_i (y_i - p(x_i))^2 over n points; coef[k] is the
 * coefficient of x^k.  w: host double[n] of weights >= 0, or NULL for all
 * ones (w_i = 1 / y_i^2 fits relative errors, for times spanning several
 * orders of magnitude).  n > degree and at least degree + 1 distinct x values
 * with positive weight; coef has degree + 1 entries.
 */
hdp_status_t hdp_fit_cost_model(const double* x, const double* y, const double* w, int32_t n, int32_t degree,
                                double* coef);

/* ====================================================================== */
/* Balance scheduler (host arithmetic only).  Research digest, section 3.4 and
 * Figure 4: micro-batches hold equal tokens but unequal attention FLOPs, so
 * workers run different numbers of them.  The section states the steps but
 * not Algorithm 2's text; the reading implemented here:
 *   1. order the micro-batches by cost, heaviest first (ties: lower index);
 *   2. cut that order into `buckets` consecutive buckets of about equal cost:
 *      the item at sorted position p goes to bucket
 *      min(B - 1, floor(B * P_p / total)), P_p the cost before it;
 *   3. HDP_BALANCE_DP: workers draw from the front of the order (the first
 *      non-empty bucket).  Each pass, every worker whose load trails the
 *      slowest worker's by more than `delta` (load + delta < max load) takes
 *      the next micro-batch, in worker order; when none trails, every worker
 *      takes one.
 *      HDP_BALANCE_PP: one bucket per pipeline (`buckets` is ignored and
 *      taken as `workers`); pipeline p runs bucket p.
 * costs: host int64[m] >= 0 (e.g. hdp_flops_per_shard copied to the host);
 * worker_of_item: host int32[m] out; worker_load: host int64[workers] out;
 * bucket_of_item: host int32[m] out, or NULL.  m >= 0, workers >= 1,
 * buckets >= 1, delta >= 0.  Time O(m log m + passes * workers); uses a
 * scratch array of m int32 allocated and freed inside the call
 * (HDP_ERR_OUT_OF_MEMORY if that fails).  The sum of the costs must fit in
 * int64. */
#define HDP_BALANCE_DP 0
#define HDP_BALANCE_PP 1
hdp_status_t hdp_balance_schedule(const int64_t* costs, int32_t m, int32_t workers, int32_t buckets, int64_t delta,
                                  int32_t mode, int32_t* worker_of_item, int64_t* worker_load,
                                  int32_t* bucket_of_item);

#ifdef __cplusplus
}
#endif

#endif /* HDPATTN_H_ */
