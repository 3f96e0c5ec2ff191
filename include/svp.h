/*
 * svp.h -- C ABI of the packed speculative-verification library (GB300, sm_103a).
 *
 * One step of block-diffusion speculative verification, as described in
 * "DScale: Scaling Block-Diffusion Speculative Decoding with Adaptive Verification"
 * (SIII-B tile routing, SIII-C Flat-buffer packer, SIII-D graph integration and Prefix
 * verifier) and the DFlash-Mini-Lab README (anchor + draft suffix, accept the exact
 * prefix, top-1/top-2 draft-logit margin):
 *
 *   N live requests; request i owns packed rows cu_slots[i] .. cu_slots[i+1]-1 of every
 *   per-row buffer; row cu_slots[i] + j holds candidate j (j = 0 is the anchor), and its
 *   target logits predict candidate j + 1.  k_i = cu_slots[i+1] - cu_slots[i] lies in
 *   [0, w] (0 = inactive).  Row j of request i attends to the request's ctx_len[i]
 *   context tokens and then to its own candidates 0..j (request-local causal mask).
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is DEVICE memory owned by the caller, unless it is marked
 *     "host".  The library never allocates, frees or synchronises; each call is
 *     enqueued on `stream` (a cudaStream_t; NULL = legacy default stream) and reads no
 *     device value back to the host, so it can be captured in a CUDA graph.
 *   - Metadata arrays (cu_slots, ctx_len, cu_ctx, block_table, cu_seqlens) are read on
 *     the device only.  Values that break the contract (cu_slots not non-decreasing,
 *     k_i > w, cu_slots[n] > m_cap, a context beyond its storage) never cause an
 *     out-of-bounds access: the affected request is skipped and a bit is set in the
 *     workspace status word (see svp_read_status).
 *   - Host-checkable errors (null pointers, head counts, unsupported head_dim or dtype,
 *     workspace too small, failed launch) are returned synchronously as svp_status and
 *     nothing is enqueued.
 *   - Workspaces: query the size, allocate it once, zero it once with
 *     svp_workspace_init, then reuse it for later calls of the same entry point.  The
 *     number of requests, m_cap and w may change from call to call (re-query the size:
 *     it grows with n); the attention workspace is tied to one head_dim and tile mode
 *     (a mismatch is reported as SVP_DEV_WORKSPACE and nothing is computed).  Kernels
 *     leave their counters and per-call scratch at zero when they finish (the attention
 *     kernel's partial slots sit at size-independent offsets before its counters), so a
 *     workspace serves later calls of any size.  Calls that share one workspace
 *     must not overlap on the GPU.  After SVP_DEV_TIMEOUT, zero the workspace again:
 *     until then an attention call on it computes nothing and reports SVP_DEV_WORKSPACE
 *     (its split-KV tickets may have been left mid-count).
 *   - Rows of out/lse that belong to no request (rows >= cu_slots[n], padding) are
 *     never written.
 *   - Kernels never trap.  Every wait inside a kernel is bounded; on expiry the kernel
 *     sets SVP_DEV_TIMEOUT in the status word and returns.
 *   - The DVL allocator, the row gathers, the verification attention, the margin /
 *     accept calls, the stochastic verifier's second pass, the cache's write and read,
 *     the chunk attention (unless the call may be a long one), the rotary positions, the
 *     pages' calls and the attention behind common pages are launched as
 *     programmatic dependents of the previous kernel on their stream: they may be
 *     scheduled while it finishes, but read nothing before it has completed, so the
 *     results are those of plain stream order (also inside a captured CUDA graph).
 */
#ifndef SVP_H_
#define SVP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SVP_VERSION 1

typedef enum {
    SVP_OK = 0,
    SVP_EINVAL = 1,          /* null pointer, negative size, hq % hkv != 0, ...        */
    SVP_EUNSUPPORTED = 2,    /* head_dim, dtype, page size or tile mode not supported  */
    SVP_EWORKSPACE = 3,      /* workspace missing or smaller than the queried size     */
    SVP_ECUDA = 4            /* a CUDA call or kernel launch failed                    */
} svp_status;

/* Bits of the device status word (svp_read_status). */
#define SVP_DEV_BAD_SLOTS   0x1   /* cu_slots decreasing, k_i > w, or cu_slots[n] > m_cap */
#define SVP_DEV_BAD_CONTEXT 0x2   /* ctx_len < 0 or a context beyond its storage          */
#define SVP_DEV_TIMEOUT     0x4   /* a bounded in-kernel wait expired                    */
#define SVP_DEV_WORKSPACE   0x8   /* workspace last used with another head_dim or tile mode:
                                     nothing was computed; run svp_workspace_init first     */
#define SVP_DEV_NO_PAGES    0x10  /* svp_pages_*: not enough free pages for all requests       */

typedef enum {
    SVP_F32 = 0,
    SVP_BF16 = 1,
    SVP_E4M3 = 2             /* paged caches only (svp_cache): 8-bit rows with an exponent byte */
} svp_dtype;

/* Query-row tile of the verification attention (DScale SIII-B, path-aware tile router). */
typedef enum {
    SVP_TILE_AUTO = 0,      /* w <= 16: SHORT, otherwise WIDE                                */
    SVP_TILE_SHORT = 1,     /* candidate-width tile: the G query heads sharing one KV head
                               are packed into one tile of G*min(w, 128/G) rows; split-KV   */
    SVP_TILE_FIXED128 = 2,  /* contrast: one query head per 128-row tile, one block per
                               (request, head), no split (the prior-art native tile)       */
    SVP_TILE_WIDE = 3,      /* prefill-style 128-row tile of one head, split-KV            */
    SVP_TILE_SHORT_UNPACKED = 4  /* contrast: the candidate-width tile without GQA packing:
                               one query head per tile of min(w, 128) rows (96 at d = 256),
                               so each KV head is streamed once per query head; split-KV;
                               d = 128 or 256                                              */
} svp_tile_mode;

/* GQA head layout.  Query head h reads KV head h / (hq / hkv). */
typedef struct {
    int32_t hq;       /* query heads                                              */
    int32_t hkv;      /* key/value heads; hq % hkv == 0                           */
    int32_t d;        /* head_dim: 64, 128 or 256                                  */
    float scale;      /* softmax scale; 0 selects 1/sqrt(d)                       */
} svp_heads;

/* Committed-context KV storage of the requests (DScale SIII-D: historyKV). */
typedef struct {
    int32_t paged;              /* 0: contiguous varlen, 1: paged                          */
    const void *k;              /* contiguous: [total_tokens, hkv, d]; paged: page pool   */
    const void *v;              /* same layout as k                                        */
    const int64_t *cu_ctx;      /* contiguous: [n] first token row of request i            */
    int64_t total_tokens;       /* contiguous: rows in k/v (a host-known allocation size) */
    const int32_t *block_table; /* paged: [n, max_pages] page ids, row-major              */
    int32_t max_pages;          /* paged: columns of block_table                          */
    int32_t page_size;          /* paged: tokens per page; must be 16                      */
    int64_t num_pages;          /* paged: pages in the pool                                */
    int64_t stride_page;        /* paged: element strides of the pool; the last dim (d)   */
    int64_t stride_head;        /*   is contiguous.  [pages][hkv][16][d] and              */
    int64_t stride_tok;         /*   [pages][16][hkv][d] are both expressible.            */
} svp_kv;

/* Library version and status text. */
int32_t svp_version(void);
const char *svp_status_string(svp_status s);

/* Zero a workspace (once, after allocating it).  Enqueued on `stream`. */
svp_status svp_workspace_init(void *ws, size_t ws_bytes, void *stream);

/* Copy the device status word of a workspace into *status (host) and clear it.
 * This is the one call that synchronises `stream`. */
svp_status svp_read_status(void *ws, void *stream, int32_t *status);

/* ---------------------------------------------------------------------------------- */
/* Verification attention over packed, ragged candidate prefixes.                      */
/* DScale SIII-B (short verify tile sized to the candidate width; grid over requests,   */
/* heads and query tiles), SIII-C (packed rows, offsets), SIII-D (rows read             */
/* offset_i + j with request-local causal masking over the supplied KV refs).           */

/* Workspace bytes for svp_verify_attn_packed(_ex) with these sizes (host). */
svp_status svp_verify_attn_workspace_size(int32_t n, int32_t m_cap, int32_t w,
                                          const svp_heads *heads, svp_dtype dtype,
                                          int32_t tile_mode, size_t *bytes);

/*
 * q      [m_cap, hq, d]   queries of the packed candidate rows
 * k_new  [m_cap, hkv, d]  keys of the packed candidate rows (same row map as q)
 * v_new  [m_cap, hkv, d]  values of the packed candidate rows
 * kv     host struct describing the committed context (contiguous or paged)
 * ctx_len  [n] int32      context tokens of each request
 * cu_slots [n+1] int32    packed row offsets (exclusive prefix sums of k_i)
 * n, m_cap, w             requests, packed row capacity, largest allowed k_i (host)
 * heads, dtype            host; q/k/v/kv/out share dtype (SVP_F32 or SVP_BF16)
 * out    [m_cap, hq, d]   softmax(scale q K^T) V per row, in dtype
 * lse    [m_cap, hq] fp32 natural-log softmax normaliser per row (may be NULL)
 * ws     workspace of at least svp_verify_attn_workspace_size bytes
 * dtype SVP_F32 runs an fp32 FFMA kernel; SVP_BF16 runs the tcgen05/TMA kernel with
 * fp32 accumulation.  All of q, k_new, v_new, kv->k, kv->v, out must be 16-byte aligned.
 */
svp_status svp_verify_attn_packed(const void *q, const void *k_new, const void *v_new,
                                  const svp_kv *kv, const int32_t *ctx_len,
                                  const int32_t *cu_slots, int32_t n, int32_t m_cap,
                                  int32_t w, const svp_heads *heads, svp_dtype dtype,
                                  void *out, float *lse, void *ws, size_t ws_bytes,
                                  void *stream);

/* As svp_verify_attn_packed, with an explicit svp_tile_mode (SVP_BF16 only for modes
 * other than AUTO). */
svp_status svp_verify_attn_packed_ex(const void *q, const void *k_new, const void *v_new,
                                     const svp_kv *kv, const int32_t *ctx_len,
                                     const int32_t *cu_slots, int32_t n, int32_t m_cap,
                                     int32_t w, const svp_heads *heads, svp_dtype dtype,
                                     int32_t tile_mode, void *out, float *lse, void *ws,
                                     size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Wide-tile causal prefill attention (the contrast path of DScale SIII-B: prefill keeps */
/* the hardware-selected 128-row tile for KV reuse).                                    */

svp_status svp_prefill_attn_workspace_size(int32_t n, int32_t max_s,
                                           const svp_heads *heads, svp_dtype dtype,
                                           size_t *bytes);

/*
 * q [total_s, hq, d], k, v [total_s, hkv, d]  sequences packed by cu_seqlens
 * cu_seqlens [n+1] int32 (device)  row offsets; sequence lengths <= max_s (host bound)
 * causal   must be 1 (SVP_EUNSUPPORTED otherwise)
 * out [total_s, hq, d] (dtype), lse [total_s, hq] fp32 (may be NULL)
 * SVP_BF16 only; 0 <= total_s < 2^31 (SVP_EINVAL otherwise).
 * Routing: d = 128 with an even number of query heads per KV head, 1 <= n <= 16 and
 *   max_s <= 32768 run the dedicated kernel (q, k, v, out 16-byte aligned, else
 *   SVP_EINVAL; it uses only the workspace header); every other shape runs the general
 *   128-row attention kernel.  A sequence whose offsets run backwards, leave the buffer or
 *   exceed max_s is skipped and sets SVP_DEV_BAD_SLOTS in the workspace status word.
 */
svp_status svp_prefill_attn(const void *q, const void *k, const void *v,
                            const int32_t *cu_seqlens, int32_t n, int32_t max_s,
                            int64_t total_s, int32_t causal, const svp_heads *heads,
                            svp_dtype dtype, void *out, float *lse, void *ws,
                            size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Row top-1 / top-2 / margin over vocabulary logits (DFlash-Mini-Lab, DFlash7-ACT     */
/* margin; DScale SII-B, Fig. 4 Top1-Top2 logit gap).                                  */
/*   top1_idx = smallest index of the row maximum; top1 = the maximum;                  */
/*   top2 = second element of the row sorted descending as a multiset (a repeated       */
/*   maximum gives top2 == top1); margin = top1 - top2 in fp32.  NaN is not supported.   */

svp_status svp_draft_margin_workspace_size(int32_t rows, int32_t vocab, size_t *bytes);

/*
 * logits [rows, row_stride] (dtype), vocab <= row_stride, vocab >= 2; rows may be 0.
 * Outputs [rows] each; any output pointer may be NULL.
 */
svp_status svp_draft_margin(const void *logits, int64_t row_stride, int32_t rows,
                            int32_t vocab, svp_dtype dtype, int32_t *top1_idx,
                            float *top1, float *top2, float *margin, void *ws,
                            size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Greedy prefix acceptance (DScale SIII-D, Prefix verifier at temperature 0;           */
/* DFlash-Mini-Lab "accept exact prefix").                                              */
/*   a_i = largest a <= k_i - 1 with tokens[off_i + j] == target_argmax[off_i + j - 1]   */
/*   for all 1 <= j <= a; accept_len[i] = 1 + a_i (the anchor counts);                   */
/*   next_token[i] = target_argmax[off_i + a_i] (row off_i + a_i supplies the successor).*/
/*   k_i = 0: accept_len = 0, next_token = -1.                                          */

/*
 * target_argmax [m_cap] int32, tokens [m_cap] int32 (row off_i = anchor, off_i + j =
 * draft j), cu_slots [n+1]; outputs accept_len [n], next_token [n].  No workspace.
 */
svp_status svp_greedy_accept(const int32_t *target_argmax, const int32_t *tokens,
                             const int32_t *cu_slots, int32_t n, int32_t m_cap,
                             int32_t *accept_len, int32_t *next_token, void *stream);

/* Fused: svp_draft_margin over the packed target-logit rows, then svp_greedy_accept,
 * in one launch.  Rows >= cu_slots[n] are not read.  m_cap rows of logits. */
svp_status svp_margin_accept_workspace_size(int32_t n, int32_t m_cap, int32_t vocab,
                                            size_t *bytes);

/*
 * logits [m_cap, row_stride] (dtype F32 or BF16, else SVP_EUNSUPPORTED): packed target
 * rows, row off_i + j the target distribution after slot j of request i; 2 <= vocab <=
 * row_stride.  tokens [m_cap] int32 (row off_i = anchor, off_i + j = draft j) and
 * cu_slots [n+1] as for svp_greedy_accept.  Outputs: top1_idx / top1 / top2 / margin
 * [m_cap] as svp_draft_margin for the live rows r < cu_slots[n] (other rows are neither
 * read nor written; any of the four pointers may be NULL); accept_len / next_token [n]
 * as svp_greedy_accept (required).  ws: at least svp_margin_accept_workspace_size bytes,
 * zeroed once by svp_workspace_init; every call leaves it zeroed.  A NULL cu_slots,
 * tokens, accept_len or next_token, n < 0, vocab < 2 or row_stride < vocab returns
 * SVP_EINVAL; a missing or small workspace SVP_EWORKSPACE; nothing is enqueued then.
 * cu_slots that break the contract on the device (not starting at 0, decreasing, or
 * cu_slots[n] > m_cap): no logit is read, no output is written and SVP_DEV_BAD_SLOTS is
 * set in the status word.
 */
svp_status svp_margin_accept(const void *logits, int64_t row_stride, int32_t m_cap,
                             int32_t vocab, svp_dtype dtype, const int32_t *tokens,
                             const int32_t *cu_slots, int32_t n, int32_t *top1_idx,
                             float *top1, float *top2, float *margin, int32_t *accept_len,
                             int32_t *next_token, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Allocation-free variant of svp_margin_accept.  The pages describe no such call; it   */
/* exists for callers that cannot allocate device memory: code running inside a memory  */
/* pool or host framework that owns every device allocation, and paths where a          */
/* cudaMalloc (and the synchronisation it may cause) is not acceptable.                 */
/*                                                                                      */
/* Arguments, outputs and results are those of svp_margin_accept, without the workspace.*/
/* The scratch is a fixed 2 MiB array inside the library, held by every GPU that loads  */
/* the library until the process exits; sizes whose workspace                           */
/* (svp_margin_accept_workspace_size) exceeds 2 MiB return SVP_EWORKSPACE and nothing   */
/* is enqueued.  The first call on each device (with that device current) looks up the  */
/* array's device address and clears it once on `stream`, waiting for that stream       */
/* (cudaGetSymbolAddress, cudaMemsetAsync, cudaStreamSynchronize; no allocation), so    */
/* make that first call before capturing any stream.  All calls share                   */
/* the one array: calls that overlap on the GPU (other streams, other host threads)     */
/* race and must be serialised by the caller.  The kernel leaves the array zeroed.      */
/* Device-side metadata errors are not reported through a status word in this variant:  */
/* invalid cu_slots leave every row and request unwritten.  Allocates nothing.          */
svp_status svp_margin_accept_noalloc(const void *logits, int64_t row_stride, int32_t m_cap,
                                     int32_t vocab, svp_dtype dtype, const int32_t *tokens,
                                     const int32_t *cu_slots, int32_t n, int32_t *top1_idx,
                                     float *top1, float *top2, float *margin,
                                     int32_t *accept_len, int32_t *next_token, void *stream);

/* ---------------------------------------------------------------------------------- */
/* DVL budget allocator and flat-buffer packer (DScale SIII-C, Budget allocator and     */
/* Flat-buffer packer, Algorithm 1, Fig. 6), one thread block, no host round trip.       */
/*   q[i,0] = 1 (anchor); q[i,j] = min(q[i,j-1], scores[i,j-1]) for j = 1..w-1.          */
/*   k0_i = clip(rint(sum_{j=1}^{w-1} q[i,j]), 1, w) for live requests (the sum in fp32, */
/*   positions in order; rint = nearest, ties to even), 0 for the others.               */
/*   budget = budget_per_req * n_live; delta = budget - sum(k0).  delta > 0: the delta   */
/*   best next slots q[i,k_i] are added (a request grows up to w); delta < 0: the -delta  */
/*   worst last slots q[i,k_i-1] are removed (never the anchor).  Ties go to the lowest   */
/*   request index.  This equals the page's one-slot-at-a-time loop because q is         */
/*   non-increasing along a request.  Growing stops when all live requests reach w,      */
/*   shrinking when all are at 1.                                                       */
/*   cu_slots = exclusive prefix sums of k (inactive requests: k = 0, offset = the end). */
/*   Packed row cu_slots[i] + j of tokens / positions / kv_refs = field[i, j] for j < k_i;*/
/*   rows cu_slots[n_bs] .. m_cap-1 hold fill_token / fill_pos / fill_ref.               */

/*
 * scores [n_bs, w-1] fp32: acceptance scores of draft positions 1..w-1 (finite; NaN not
 * supported).  n_live: device int32 scalar (requests 0..n_live-1 are live), or NULL for
 * all n_bs.  tokens / positions / kv_refs [n_bs, w] int32, each may be NULL (then the
 * matching packed output is all fill, or not written if its pointer is NULL too).
 * Outputs: k_init [n_bs] (may be NULL), k_out [n_bs], cu_slots [n_bs + 1],
 * tokens_packed / pos_packed / ref_packed [m_cap] (each may be NULL), n_adjust (device
 * int32 scalar, slots added or removed; may be NULL).  ws: at least 256 bytes, zeroed
 * once (svp_workspace_init); n_live outside [0, n_bs] or budget > m_cap sets
 * SVP_DEV_BAD_SLOTS and treats every request as inactive.
 * Limits: 1 <= n_bs <= 2048, 2 <= w <= 16, 1 <= budget_per_req <= w, m_cap >= 1
 * (SVP_EINVAL / SVP_EUNSUPPORTED otherwise).
 */
svp_status svp_dvl_allocate_pack(const float *scores, int32_t n_bs, int32_t w,
                                 const int32_t *n_live, int32_t budget_per_req,
                                 const int32_t *tokens, const int32_t *positions,
                                 const int32_t *kv_refs, int32_t m_cap, int32_t fill_token,
                                 int32_t fill_pos, int32_t fill_ref, int32_t *k_init,
                                 int32_t *k_out, int32_t *cu_slots, int32_t *tokens_packed,
                                 int32_t *pos_packed, int32_t *ref_packed, int32_t *n_adjust,
                                 void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Row-mapped packing of a wide per-row field (DScale SIII-C, Flat-buffer packer: every  */
/* field is packed with the same row mapping; SIII-D, fixed-address workspace).          */
/*   dst row r = src row idx[r] for 0 <= idx[r] < src_rows, else zeros; r < rows.       */

/*
 * src [src_rows, row_bytes] and dst [rows, row_bytes] device buffers, 16-byte aligned,
 * row_bytes >= 16 (SVP_EINVAL otherwise, as for NULL pointers or negative counts) and a
 * multiple of 16 (SVP_EUNSUPPORTED otherwise, as for unaligned buffers); idx [rows] int32
 * (e.g. the packed KV references of svp_dvl_allocate_pack).  No workspace.
 */
svp_status svp_gather_rows(const void *src, int64_t src_rows, int64_t row_bytes,
                           const int32_t *idx, int32_t rows, void *dst, void *stream);

/*
 * The same for up to SVP_GATHER_MAX_FIELDS fields that share one row map, in one launch
 * (a step packs its query, key, value and logit rows together).  fields: a HOST array of
 * n_fields descriptors (1 <= n_fields <= SVP_GATHER_MAX_FIELDS), read during the call and
 * not retained, SVP_EINVAL for a count outside that range; each src / dst pair follows
 * the rules of svp_gather_rows (16-byte aligned, row_bytes >= 16 and a multiple of 16);
 * dst of field f holds [rows, row_bytes_f].  idx [rows] int32, shared.  No workspace.
 */
#define SVP_GATHER_MAX_FIELDS 8
typedef struct {
    const void *src;    /* [src_rows, row_bytes] */
    int64_t src_rows;
    int64_t row_bytes;
    void *dst;          /* [rows, row_bytes] */
} svp_gather_field;

svp_status svp_gather_rows_multi(const svp_gather_field *fields, int32_t n_fields,
                                 const int32_t *idx, int32_t rows, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Stochastic prefix verifier, temperature T > 0 (DScale SIII-D, Prefix verifier).       */
/*   P_r = softmax(logits[r] / T).  Candidate j of request i (tokens[off_i + j],          */
/*   1 <= j < k_i) is accepted iff u_accept[off_i + j] < P_{off_i+j-1}(candidate), in     */
/*   order; the first rejection ends the prefix.  a_i = accepted candidates;              */
/*   accept_len[i] = 1 + a_i.  The successor next_token[i] is the smallest token y with   */
/*   sum_{y' <= y} w(y') > u_next[i] * sum w, over row off_i + a_i with weights          */
/*   w = P_{off_i+a_i}, the rejected candidate's weight set to 0 (none removed when every */
/*   candidate passed).  k_i = 0: accept_len 0, next_token -1.  The row softmax is       */
/*   evaluated in fp32 (exp2 of scaled differences), so a draw within rounding of a      */
/*   boundary may fall on either side.                                                    */

svp_status svp_stochastic_accept_workspace_size(int32_t m_cap, int32_t vocab, size_t *bytes);

/*
 * logits [m_cap, row_stride] (dtype), vocab <= row_stride; tokens [m_cap] int32;
 * cu_slots [n+1]; u_accept [m_cap] fp32 and u_next [n] fp32, uniform draws in [0, 1)
 * supplied by the caller; outputs accept_len [n], next_token [n] int32 and p_draft [m_cap]
 * (the acceptance probability of each tested candidate; may be NULL).  Rows >=
 * cu_slots[n] are not read.  Invalid cu_slots (cu_slots[0] != 0, a decrease, or
 * cu_slots[n] > m_cap) set SVP_DEV_BAD_SLOTS: no row is read and every request gets
 * accept_len 0 and next_token -1.  ws zeroed once (svp_workspace_init); the kernels leave
 * it zeroed (tickets, row and chunk statistics), so it can serve later calls with other
 * m_cap and vocabularies.
 */
svp_status svp_stochastic_accept(const void *logits, int64_t row_stride, int32_t m_cap,
                                 int32_t vocab, svp_dtype dtype, const int32_t *tokens,
                                 const int32_t *cu_slots, int32_t n, float temperature,
                                 const float *u_accept, const float *u_next,
                                 int32_t *accept_len, int32_t *next_token, float *p_draft,
                                 void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Draft-signal features (DScale SIII-C, Acceptance predictor).  For every row of draft  */
/* logits, 18 fp32 values: [0] the highest logit; [1..15] its gaps to ranks 2..16 (rank r */
/* = r-th element of the row sorted descending as a multiset, gap = top1 - rank_r in     */
/* fp32); [16] the top token's log-probability (top1 - log-sum-exp of the row); [17] the  */
/* entropy -sum p ln p of softmax(row).  Sums are fp32.                                    */

svp_status svp_draft_features_workspace_size(int32_t rows, int32_t vocab, size_t *bytes);

/*
 * logits [rows, row_stride] (dtype), 16 <= vocab <= row_stride; features [rows, 18] fp32.
 * ws zeroed once (svp_workspace_init); the kernel leaves it zeroed (tickets and partial
 * lists), so it can serve later calls with other row counts and vocabularies.
 */
svp_status svp_draft_features(const void *logits, int64_t row_stride, int32_t rows,
                              int32_t vocab, svp_dtype dtype, float *features, void *ws,
                              size_t ws_bytes, void *stream);

/* ACT truncation (DFlash-Mini-Lab README, DFlash7-ACT): the draft suffix of request i is  */
/* cut before its first position j (1 <= j < w) whose margin is below `threshold`;       */
/* k_out[i] = 1 + the number of positions kept (threshold 0 keeps the full block w).      */
/* margins: element ((i * (w-1) + j - 1) * stride) is the margin of position j of request */
/* i (stride = 1 for svp_draft_margin's margin array, 18 with features + 1).  No         */
/* workspace.                                                                             */
svp_status svp_act_truncate(const float *margins, int64_t stride, int32_t n, int32_t w,
                            float threshold, int32_t *k_out, void *stream);

/* ---------------------------------------------------------------------------------- */
/* The paged cache's own calls: writing new key / value rows into the pages (the rows of */
/* a prompt, of a decode step, or the accepted candidates after a verification), reading */
/* cached positions back to contiguous rows, and attention of a chunk of new tokens      */
/* whose keys and values are already in the pages.                                       */
/*                                                                                      */
/* 8-bit rows (SVP_E4M3): the d elements of one token and head are e4m3 codes with one   */
/* exponent byte b; an element is code * 2^(b - 127).  svp_cache_write picks the smallest */
/* power of two that takes the row's largest magnitude to 448 or less (b >= 15), so        */
/* scaling is exact and each element is rounded once, to nearest even: at most 2^-4       */
/* relative for elements down to 2^-13 of the row's largest (2^-6 of that power or more;  */
/* smaller ones round to a multiple of 2^-9 of it).  A row with an infinite or NaN        */
/* element gets b = 255 and codes 0: every element of it reads as NaN, as do codes 0x7f   */
/* and 0xff.  Readers take any byte (b = 0 as 0).                                         */
typedef struct {
    void *k, *v;                /* page pools, [num_pages] pages of page_size tokens; 16-byte
                                   aligned                                                 */
    uint8_t *k_exp, *v_exp;     /* SVP_E4M3: exponent bytes [num_pages, hkv, page_size],
                                   16-byte aligned; else NULL                              */
    const int32_t *block_table; /* device [n, max_pages] page ids, row-major               */
    int32_t max_pages;          /* columns of block_table                                  */
    int32_t page_size;          /* tokens per page: 16, 32, 64 or 128                      */
    int64_t num_pages;          /* pages in the pool, < 2^31                               */
    int64_t stride_page;        /* element strides of both pools, multiples of 16 bytes;   */
    int64_t stride_head;        /*   the last dim (d) is contiguous, and no two (page,      */
    int64_t stride_tok;         /*   head, token) rows overlap                             */
    svp_dtype dtype;            /* SVP_F32, SVP_BF16 or SVP_E4M3                           */
} svp_cache;

/*
 * Row j of request i (packed row cu_slots[i] + j of k and v) goes to position ctx_len[i] + j
 * of the request, i.e. to page block_table[i][pos / page_size], token pos % page_size.
 * k, v      rows [m_cap, hkv, d] (dtype SVP_F32 or SVP_BF16), row r at element r * row_stride
 *           (row_stride >= hkv * d, so both may be slices of a fused projection's output);
 *           16-byte aligned, row_stride a multiple of 16 bytes
 * ctx_len   [n] int32; cu_slots [n+1] int32
 * take      [n] int32 or NULL: only rows j < take[i] are written (clamped to 0..k_i), e.g. the
 *           accept_len of svp_greedy_accept / svp_margin_accept / svp_stochastic_accept
 * ws        at least 256 bytes, zeroed once by svp_workspace_init (status word only)
 * Rows >= cu_slots[n] may be read but are not used.  An SVP_F32 row is rounded to nearest
 * even for an SVP_BF16 cache.  A request whose rows leave [0, m_cap) or run backwards is
 * skipped (SVP_DEV_BAD_SLOTS); one with ctx_len < 0 or positions past max_pages * page_size is
 * skipped, and a row whose page id is outside [0, num_pages) is not written
 * (SVP_DEV_BAD_CONTEXT).  Two rows of one call must not share a (page, token).
 */
svp_status svp_cache_write(const void *k, const void *v, int64_t row_stride, svp_dtype dtype,
                           const svp_cache *cache, const int32_t *ctx_len,
                           const int32_t *cu_slots, const int32_t *take, int32_t n,
                           int32_t m_cap, int32_t hkv, int32_t d, void *ws, size_t ws_bytes,
                           void *stream);

/*
 * The inverse: row cu_rows[i] + j of k_out / v_out [rows, hkv, d] (dtype SVP_F32 or SVP_BF16,
 * contiguous, 16-byte aligned) = position start[i] + j of request i, 0 <= j < cu_rows[i+1] -
 * cu_rows[i].  start [n] int32, or NULL for 0.  Values of an 8-bit row are exact in both types
 * (bf16: while the product is a normal bf16 number).  Other rows of the outputs are left as
 * they were.  Errors, status bits and ws as for svp_cache_write; a row whose page id is
 * invalid is not written.  The output is the contiguous context of svp_verify_attn_packed.
 */
svp_status svp_cache_read(const svp_cache *cache, const int32_t *start, const int32_t *cu_rows,
                          int32_t n, int32_t rows, int32_t hkv, int32_t d, svp_dtype dtype,
                          void *k_out, void *v_out, void *ws, size_t ws_bytes, void *stream);

/*
 * Attention of new tokens over the pages: row j of request i (packed row cu_slots[i] + j) sees
 * positions 0 .. ctx_len[i] + j of its request, all of them in the cache (svp_cache_write puts
 * the rows' own keys and values there first).  One call serves decode tokens (k_i = 1),
 * candidate blocks and prompt chunks of thousands of rows together.
 *   out = softmax(scale q K^T) V, lse = natural-log softmax normaliser (may be NULL)
 * q      [m_cap, hq, d], row r at element r * q_row_stride (>= hq * d; 16-byte aligned, a
 *        multiple of 16 bytes); out [m_cap, hq, d] contiguous, lse [m_cap, hq] fp32
 * w      largest allowed k_i (host; 1 <= w); a request with k_i > w is skipped
 * heads  scale 0 selects 1/sqrt(d); a negative, infinite or NaN one is SVP_EINVAL
 * dtype  of q and out: SVP_BF16 with an SVP_BF16 or SVP_E4M3 cache, SVP_F32 with an SVP_F32
 *        cache (anything else: SVP_EUNSUPPORTED)
 * ws     at least svp_chunk_attn_workspace_size bytes (it depends on d and dtype only), its
 *        first 256 zeroed once by svp_workspace_init; every call leaves it ready for the next
 *        one of any size, head layout or type that it is large enough for; 32-byte aligned with
 *        SVP_BF16 (SVP_EINVAL otherwise)
 * 0 <= n <= 1024, hq / hkv <= 128, d = 64, 128 or 256 (SVP_EUNSUPPORTED otherwise).
 *
 * Precision.  Scores, the softmax's maximum and sum, and the output are accumulated in fp32; the
 * probabilities that multiply V are rounded to bf16 over SVP_BF16 pages and to fp16 over SVP_E4M3
 * ones (not at all in fp32), where one (times the power of two of its value row, or of its tile,
 * see below) under 2^-21 of the row's largest has fewer digits and one under 2^-32 counts in the
 * sum only.  8-bit rows with hq / hkv * w <= 16 and d <= 128 are used as they are; otherwise 128
 * positions (a tile) at a time in units of their largest power of two 2^E (of K and of V each, of
 * visible rows, at least 2^-60): exact for rows within 2^15 of it, and an element of 2^(E - 25) or
 * less counts as 0.  8-bit value rows of one request should have powers of two within 2^100 of one
 * another (rows of zeros count as 2^-60 whatever their byte): beyond, a key's weight can be lost.
 * lse takes nothing from the values: it is finite where they are NaN.
 *
 * Rows >= cu_slots[n] and rows of skipped requests are not written.  Device checks as for
 * svp_cache_write, for positions 0 .. ctx_len[i] + k_i - 1; a page id outside the pool reads
 * as a page of zeros (SVP_DEV_BAD_CONTEXT).  Cache positions past a request's last row (the
 * rest of its last page) may hold anything, NaN included; a NaN or infinity in the value row
 * of a position that some row of the request may not see yet can reach that row.
 */
svp_status svp_chunk_attn_workspace_size(const svp_heads *heads, svp_dtype dtype, size_t *bytes);

svp_status svp_chunk_attn(const void *q, int64_t q_row_stride, const svp_cache *cache,
                          const int32_t *ctx_len, const int32_t *cu_slots, int32_t n,
                          int32_t m_cap, int32_t w, const svp_heads *heads, svp_dtype dtype,
                          void *out, float *lse, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* Rotary positions for the rows of a step, and the same together with the cache's write.  */
/*   pos = ctx_len[i] + j of row j of request i (or pos[row]);  pair t < rot / 2 of a head   */
/*   turns by the angle 2 pi pos freq[t] / 2^64:                                            */
/*     (x, y) -> scale (x cos - y sin, x sin + y cos)                                       */
/*   with (x, y) = elements (t, t + rot / 2), or (2 t, 2 t + 1) when interleaved.  Elements   */
/*   from rot on stay as they are.  pos * freq is taken modulo 2^64, i.e. whole turns drop   */
/*   out exactly, so far positions lose nothing; sine, cosine and the products are fp32.     */
/*   Negative positions turn back: rows rotated at pos and then at -pos are the rows again   */
/*   (but for their roundings), which is also the gradient's way back.                       */
typedef enum {
    SVP_ROPE_NONE = 0,       /* base^(-2t / rot) radians a position                         */
    SVP_ROPE_LINEAR = 1,     /* divided by factor (positions interpolated)                  */
    SVP_ROPE_NTK = 2,        /* base * factor^(rot / (rot - 2)) in base's place             */
    SVP_ROPE_YARN = 3        /* pairs that turn more than `fast` times in `original` tokens
                                as NONE, those that turn less than `slow` times as LINEAR, a
                                straight line (in t) between.  That method's factor on the
                                scores, 0.1 ln(factor) + 1 on q and k each, is `scale`.      */
} svp_rope_scaling;

/* Fills freq[0 .. rot / 2 - 1] (HOST memory): turns a position in units of 2^-64, from 64-bit
 * radians.  rot even and >= 2, base > 1, factor > 0; YARN: original >= 1, 0 < slow < fast
 * (SVP_EINVAL otherwise).  For SVP_ROPE_NTK rot = 2 has nothing to change. */
svp_status svp_rope_frequencies(int32_t rot, double base, svp_rope_scaling scaling, double factor,
                                int32_t original, double slow, double fast, uint64_t *freq);

typedef struct {
    const uint64_t *freq;    /* device [rot / 2]                                            */
    int32_t rot;             /* elements of a head that turn: even, 2 <= rot <= d           */
    int32_t interleaved;     /* 0: pairs (t, t + rot / 2), 1: (2 t, 2 t + 1)                 */
    float scale;             /* on the elements that turn; finite                           */
} svp_rotary;

/*
 * q [m_cap, hq, d], k [m_cap, hkv, d] (dtype SVP_F32 or SVP_BF16), row r at element r * row
 * stride (slices of a fused projection); q_out, k_out of the same type and shape with strides of
 * their own.  An output may be its input itself (the same address and stride); otherwise no output
 * overlaps an input or another output.  q and q_out, or k and k_out, may be NULL (hq or hkv is then
 * not looked at).  All 16-byte aligned, strides >= heads * d and multiples of 16 bytes.
 * pos [m_cap] int32 or NULL; ctx_len [n] int32 (NULL only with pos); cu_slots [n+1] int32
 * ws at least 256 bytes, zeroed once by svp_workspace_init (status word only)
 * d = 64, 128 or 256.  Rows of no request are not written.  A request whose rows leave [0, m_cap) or
 * run backwards is skipped (SVP_DEV_BAD_SLOTS), without pos one with ctx_len < 0 or positions past
 * 2^31 - 1 too (SVP_DEV_BAD_CONTEXT).
 */
svp_status svp_rope(const void *q, int64_t q_row_stride, const void *k, int64_t k_row_stride,
                    svp_dtype dtype, const svp_rotary *rotary, const int32_t *pos,
                    const int32_t *ctx_len, const int32_t *cu_slots, int32_t n, int32_t m_cap,
                    int32_t hq, int32_t hkv, int32_t d, void *q_out, int64_t q_out_stride,
                    void *k_out, int64_t k_out_stride, void *ws, size_t ws_bytes, void *stream);

/*
 * svp_rope for q (NULL: none) and k, with the rotated k and v written to the cache as
 * svp_cache_write does (positions ctx_len[i] + j, take, types, errors and status bits are its own;
 * pos, where given, is for the angles only).  k goes from fp32 to the cache's type in one rounding.
 * A request that svp_cache_write skips is skipped for q too; rows behind take[i] are rotated in q.
 */
svp_status svp_rope_cache_write(const void *q, int64_t q_row_stride, const void *k, const void *v,
                                int64_t kv_row_stride, svp_dtype dtype, const svp_rotary *rotary,
                                const svp_cache *cache, const int32_t *pos, const int32_t *ctx_len,
                                const int32_t *cu_slots, const int32_t *take, int32_t n,
                                int32_t m_cap, int32_t hq, int32_t hkv, int32_t d, void *q_out,
                                int64_t q_out_stride, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------------- */
/* The pages of a cache: who holds them, and their sharing, freeing and moving, all on the */
/* device (no host round trip, so a captured step may allocate).                           */
/*   block_table [n, max_pages]: entries 0 .. used[i] - 1 of row i are request i's pages.   */
/*   refs [num_pages]: how many entries hold a page; 0 means free.                         */
/* To start: refs and used 0 (then every page is free), and resize the requests.  A page   */
/* shared by several requests is read by all and written by none: every request's last,    */
/* partly filled page stays its own, see svp_pages_fork and svp_pages_resize.              */
typedef struct {
    int32_t *block_table;    /* device [n, max_pages], the block_table of svp_cache         */
    int32_t *used;           /* device [n]                                                  */
    int32_t *refs;           /* device [num_pages]                                          */
    int32_t n, max_pages;    /* 0 <= n <= 1024                                              */
    int32_t page_size;       /* tokens per page: 16, 32, 64 or 128                          */
    int64_t num_pages;       /* < 2^31                                                      */
} svp_pages;

#define SVP_PAGES_MAX_CACHES 64

/* Workspace bytes for the three calls below (host; grows with num_pages). */
svp_status svp_pages_workspace_size(const svp_pages *pages, size_t *bytes);

/*
 * Request i ends with ceil(length[i] / page_size) pages (length [n] int32, device; a negative one
 * leaves the request as it is): before a step that writes up to ctx_len + k_i, after an acceptance that
 * kept fewer, with 0 when it is done.  First every shrinking request gives back its pages from the end
 * (refs - 1, entries -1); then the growing ones get the free pages with the lowest ids, in the order
 * of requests and positions (refs 1).  Without enough free pages a request i is left as it was when what
 * requests 0 .. i ask for together is more than there are (SVP_DEV_NO_PAGES).
 * Left as they were too (SVP_DEV_BAD_CONTEXT): a request with used[i] outside 0 .. max_pages, a length
 * past max_pages * page_size, and one that would end in a part of a page of its own that another holds as well
 * (refs > 1 before the call), as its next write would go there: give it a whole page less, or fork it instead.
 * An entry that names no page of the pool, or one whose refs is 0 already, is given back as -1 without
 * counting (SVP_DEV_BAD_CONTEXT).
 * ws     at least svp_pages_workspace_size bytes, its first 256 zeroed once by svp_workspace_init; 16-byte aligned
 */
svp_status svp_pages_resize(const svp_pages *pages, const int32_t *length, void *ws,
                            size_t ws_bytes, void *stream);

/*
 * Request dst[f], which holds no page, gets the first length[f] tokens of src[f] (0 <= f < forks;
 * int32 [forks], device): the whole pages among them are shared (refs + 1), and a part of a page at the
 * end is copied, its tokens only, to a page of its own (refs 1): the lowest free ids in the order of f.
 * The length[f] tokens are ones that src[f] has written and will not write again.
 * caches: HOST array of the n_caches <= SVP_PAGES_MAX_CACHES caches (a model's layers) that this block
 * table serves, of one type, strides, page size and num_pages, hkv heads of d; read during the call and
 * not retained.  n_caches may be 0 (the caller copies).  The rest of block_table's row dst[f] is -1.
 * Not done: a src or dst outside 0 .. n - 1, a dst that holds pages or is that of an earlier fork of the
 * call (SVP_DEV_BAD_SLOTS); a length outside 0 .. used[src] * page_size (SVP_DEV_BAD_CONTEXT); a fork when
 * forks 0 .. f together need more pages than are free (SVP_DEV_NO_PAGES).  An entry of src that names no
 * page of the pool is passed on as -1 (SVP_DEV_BAD_CONTEXT), that of the part at the end too, for which no page is
 * taken then.  0 <= forks <= 1024, hkv <= 4096.
 */
svp_status svp_pages_fork(const svp_pages *pages, const svp_cache *caches, int32_t n_caches,
                          int32_t hkv, int32_t d, const int32_t *src, const int32_t *dst,
                          const int32_t *length, int32_t forks, void *ws, size_t ws_bytes,
                          void *stream);

/*
 * Moves pages so that the L pages in use (refs other than 0) are pages 0 .. L - 1: of those with
 * ids >= L, in their order, the k-th goes to the k-th free id below L, with its contents in every cache, its
 * refs and every entry that holds it.  live: device int32 that gets L, or NULL.  Pages >= L are free
 * then (and hold what they held).  An entry that holds a page with refs 0 is left as it is
 * (SVP_DEV_BAD_CONTEXT when its id is >= L).  caches as above.
 */
svp_status svp_pages_compact(const svp_pages *pages, const svp_cache *caches, int32_t n_caches,
                             int32_t hkv, int32_t d, int32_t *live, void *ws, size_t ws_bytes,
                             void *stream);

/* ---------------------------------------------------------------------------------- */
/* Attention of requests that share a beginning (samples of one prompt, a common system    */
/* prompt; svp_pages_fork makes such requests).                                            */
/*
 * The result is svp_chunk_attn's, argument by argument; in addition, requests cu_groups[g] ..
 * cu_groups[g+1] - 1 form group g (requests outside all groups are alone), and the first prefix_len[g]
 * tokens of each of them lie in the same pages: the block table's rows of a group's requests (of
 * those with k_i > 0) have the same ids there, and only the first one's are read.  The whole pages of a
 * prefix are read once for 256 / (hq / hkv) rows of the group (128 / (hq / hkv) at d = 256) instead of once
 * for every request, where that is fewer times.  The call is for long prefixes: where they are short beside the
 * requests' own contexts, for a few decode tokens over 8-bit pages and for prompt chunks svp_chunk_attn is the quicker one.
 * cu_groups [n_groups+1], prefix_len [n_groups] int32 (device); 0 <= n_groups <= 1024
 * With an SVP_F32 cache, or without groups, the call is svp_chunk_attn (groups are not looked at).
 * ws     at least svp_prefix_attn_workspace_size bytes (it grows with m_cap), its first 256 zeroed once by
 *        svp_workspace_init; every call leaves it ready for the next one that it is large enough for; 32-byte
 *        aligned with SVP_BF16 (SVP_EINVAL otherwise)
 * Device checks are svp_chunk_attn's, but cu_slots that run backwards or leave [0, m_cap] anywhere reject the
 * whole call (SVP_DEV_BAD_SLOTS; nothing is written).  Groups that run backwards or leave [0, n] anywhere are
 * none (SVP_DEV_BAD_SLOTS), and a group with prefix_len < 0 or > the ctx_len of a member with rows
 * (SVP_DEV_BAD_CONTEXT), or with a member that is skipped, is not shared; its other requests then use their own entries.
 * Precision and values: as svp_chunk_attn's.  8-bit rows of a shared prefix are in units of their tile's largest power
 * of two whatever w is, and a request's own ones unless hq / hkv * w <= 8 and d <= 128, where they are used as they
 * are.  A row's two parts stay in fp32 until they are joined.
 */
svp_status svp_prefix_attn_workspace_size(const svp_heads *heads, svp_dtype dtype, int32_t m_cap,
                                          size_t *bytes);

svp_status svp_prefix_attn(const void *q, int64_t q_row_stride, const svp_cache *cache,
                           const int32_t *ctx_len, const int32_t *cu_slots, int32_t n,
                           int32_t m_cap, int32_t w, const int32_t *cu_groups,
                           const int32_t *prefix_len, int32_t n_groups, const svp_heads *heads,
                           svp_dtype dtype, void *out, float *lse, void *ws, size_t ws_bytes,
                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVP_H_ */
