/*
 * orthros_attn.h -- C ABI of the Orthros attention hot path on one GPU.
 *
 * Orthros ("Orthros: Phase-Aware Heterogeneous Attention for Efficient
 * Transformers", paperz.arrangedbits.com full text) runs, in every layer:
 *   - a base stream: sliding-window attention of EVERY position t over the keys
 *     max(0, t-w+1) .. t  (Sec. 3.1, Eq. 4; 0-indexed here), which also
 *     produces the layer's K/V cache;
 *   - an output stream: full causal cross-attention of the output positions
 *     over keys 0 .. t of the same K/V (Sec. 3.1, Eq. 5).
 * Both query streams come from one Q projection through their own
 * per-channel scale-offset affine, q = alpha (.) q_raw + beta (Sec. 3.1,
 * Alg. 1 line 5). The four regimes of Sec. 3.2 (pre-training, SFT,
 * prefilling, decoding) differ only in which positions are output rows.
 *
 * Conventions shared by every entry point
 *   - All tensor arguments are DEVICE pointers unless marked HOST. The caller
 *     owns every buffer, including the workspace and the cache pages; the
 *     library never allocates, frees or synchronises on the compute path.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = default stream).
 *   - Layouts are row-major and contiguous. Query heads h map to K/V heads
 *     kv = h / (Hq / Hkv) (contiguous groups; Hq == Hkv is plain multi-head).
 *   - Element type of q, k, v, q_out, k_new, v_new, caches and o_* is given by
 *     `dtype`: ORTHROS_BF16 (bfloat16) or ORTHROS_F32 (float). alpha/beta and
 *     lse are always float. lse is the natural log of sum_j exp(scale q.k_j).
 *   - The logit is scale * (q_affined . k); scale is usually 1/sqrt(d)
 *     (Sec. 2.1, Eq. 1).
 *   - Tensors of element type bf16/f32 must be 16-byte aligned.
 *   - Errors found on the host return before any launch (ORTHROS_EINVAL,
 *     ORTHROS_EUNSUPPORTED, ORTHROS_EWORKSPACE); orthros_last_error() then
 *     describes the problem. Launch failures return ORTHROS_ECUDA. Bad data
 *     that only the GPU can see (a position out of range, a block-table entry
 *     outside the page pool, a cache length past the block table) sets a
 *     status word in the
 *     workspace; the affected rows are skipped or their outputs are NaN, and
 *     orthros_check() reports ORTHROS_EDEVICE. Nothing aborts or traps.
 *   - Supported head sizes: d = 64 or 128.
 *   - The *_workspace_size functions size the scratch for the CUDA device that
 *     is current when they are called (the split-KV partials depend on its SM
 *     count); call them with the device that will run the call current. A
 *     workspace smaller than the call then needs returns ORTHROS_EWORKSPACE.
 */
#ifndef ORTHROS_ATTN_H
#define ORTHROS_ATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ORTHROS_API __attribute__((visibility("default")))
#else
#define ORTHROS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *orthros_stream_t; /* same type as cudaStream_t */

typedef enum {
    ORTHROS_OK = 0,
    ORTHROS_EINVAL = 1,       /* bad argument, detected on the host */
    ORTHROS_EUNSUPPORTED = 2, /* well-formed but not supported (e.g. d = 96) */
    ORTHROS_ECUDA = 3,        /* a CUDA call or kernel launch failed */
    ORTHROS_EWORKSPACE = 4,   /* workspace NULL or smaller than required */
    ORTHROS_EDEVICE = 5,      /* a kernel flagged bad device-side data */
    ORTHROS_ETIMEOUT = 6      /* a kernel's bounded wait ran out */
} orthros_status;

typedef enum { ORTHROS_BF16 = 0, ORTHROS_F32 = 1 } orthros_dtype;

/* Bits of the device status word (see orthros_check). */
#define ORTHROS_DEV_BAD_POSITION 0x1u  /* out_positions entry outside [0, T) */
#define ORTHROS_DEV_BAD_PAGE 0x2u      /* block-table entry outside [0, num_pages) */
#define ORTHROS_DEV_BAD_LENGTH 0x4u    /* cache_lens[b] < 0 or past the block table */
/* 0x8u is never raised: keys and affined queries beyond the fp16 range of the
 * tensor-core prefill are scaled by exact powers of two (the logit scale
 * takes the inverse), so any finite bf16 input is served. */
#define ORTHROS_DEV_FP16_RANGE 0x8u
#define ORTHROS_DEV_TIMEOUT 0x10u      /* a bounded wait inside a kernel ran out */
#define ORTHROS_DEV_NO_PAGES 0x20u     /* a step needs more pages than are free */

/*
 * Workspace bytes orthros_prefill needs for these sizes. n_out is the total
 * number of output rows. Returns 0 for sizes orthros_prefill would reject.
 */
ORTHROS_API size_t orthros_prefill_workspace_size(int B, int T, int Hq, int Hkv, int d,
                                      int n_out, int window, orthros_dtype dtype);

/*
 * Prefill (Sec. 3.2 regimes pre-training / SFT / prefilling): Eq. 4 at every
 * position of B sequences of T tokens, Eq. 5 at the output rows, and
 * optionally the paged K/V cache fill that the decoding phase reads.
 *
 * q            [B, T, Hq, d]   raw queries (the affines are applied inside)
 * k, v         [B, T, Hkv, d]
 * alpha_base, beta_base [Hq, d] float: base-stream affine (alpha, beta)
 * alpha_out,  beta_out  [Hq, d] float: output-stream affine (alpha', beta');
 *              may be NULL when n_out == 0
 * out_indptr   HOST [B+1] int32, out_indptr[0] = 0, non-decreasing,
 *              out_indptr[B] = n_out: output rows of sequence b are
 *              r in [out_indptr[b], out_indptr[b+1])
 * out_positions [n_out] int32: position t_r in [0, T) of output row r (any
 *              order, repeats allowed; each row is independent)
 * q_out        [n_out, Hq, d] raw output-stream queries, or NULL: then the raw
 *              query of row r is q[b, t_r] (one shared Q projection; exact for
 *              a first layer, whose output tokens duplicate the base tokens)
 * window       w >= 1; w >= T gives full causal attention in the base stream
 * scale        logit scale (finite)
 * o_base [B, T, Hq, d], lse_base [B, Hq, T] float
 * o_out  [n_out, Hq, d], lse_out [n_out, Hq] float  (may be NULL if n_out == 0)
 * k_cache, v_cache [num_pages, page_size, Hkv, d], block_table [B, max_pages]
 *              int32: optional (all NULL to skip). When given, token t of
 *              sequence b is also written to page block_table[b*max_pages +
 *              t/page_size], slot t % page_size, for t < T (needs
 *              max_pages * page_size >= T). num_pages bounds the entries.
 * workspace    device scratch of at least orthros_prefill_workspace_size()
 *              bytes, 256-byte aligned; its contents on entry do not matter.
 */
ORTHROS_API orthros_status orthros_prefill(
    const void *q, const void *k, const void *v,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    const int32_t *out_indptr, const int32_t *out_positions, int n_out,
    const void *q_out,
    int B, int T, int Hq, int Hkv, int d, int window, float scale,
    orthros_dtype dtype,
    void *o_base, float *lse_base, void *o_out, float *lse_out,
    void *k_cache, void *v_cache, const int32_t *block_table,
    int max_pages, int page_size, int num_pages,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/* Workspace bytes orthros_prefill_from_host needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_prefill_from_host_workspace_size(int B, int T, int Hq, int Hkv, int d, int n_out,
                                                            int window, orthros_dtype dtype);

/*
 * orthros_prefill with the step's inputs and outputs in HOST memory: the
 * same computation (Eq. 4 for every position, Eq. 5 for the output rows, the
 * optional cache fill), the host-to-device and device-to-host copies included.
 *
 * HOST:   q, k, v, o_base, lse_base, out_indptr, out_positions, q_out, o_out,
 *         lse_out, with the shapes of orthros_prefill. Page-locked memory
 *         (cudaHostAlloc / cudaHostRegister) lets the copies overlap the
 *         compute; pageable memory gives the same results with copies that do
 *         not overlap. Device memory passed here is rejected (ORTHROS_EINVAL).
 * DEVICE: alpha_base, beta_base, alpha_out, beta_out (model parameters), the
 *         optional k_cache, v_cache, block_table, and the workspace (at least
 *         orthros_prefill_from_host_workspace_size() bytes, 256-byte aligned;
 *         it holds device copies of q, k, v and o_base besides the scratch).
 * out_positions are checked on the host: a position outside [0, T) returns
 * ORTHROS_EINVAL before anything is enqueued.
 *
 * A sequence longer than one chunk (at least 16384 tokens and four halos of
 * w - 1 keys; bf16 only) is computed chunk by chunk as orthros_prefill_shard
 * calls (each chunk's keys with the halo before it, so its base rows are
 * exact, and each output row's partial over the chunk's keys), and the
 * partials are merged as orthros_merge_partials does, so the results equal
 * orthros_prefill's up to the rounding of that merge. Chunk c + 1 is copied
 * in while chunk c computes and chunk c - 1 is copied out, on two copy streams
 * of the library's own (created once per device) ordered after the work
 * already on `stream`; `stream` itself runs the compute and waits for the
 * last copy out, so every output is in host memory once `stream` reaches the
 * point after this call (also after an error return: what the call had
 * already enqueued on its copy streams is joined to `stream`). Calls are
 * enqueued one at a time (an internal lock).
 * Shorter sequences, and f32, copy everything in, compute, and copy out on
 * `stream`. Device-side status as for orthros_prefill (orthros_check on this
 * call's workspace).
 */
ORTHROS_API orthros_status orthros_prefill_from_host(
    const void *q, const void *k, const void *v,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    const int32_t *out_indptr, const int32_t *out_positions, int n_out,
    const void *q_out,
    int B, int T, int Hq, int Hkv, int d, int window, float scale,
    orthros_dtype dtype,
    void *o_base, float *lse_base, void *o_out, float *lse_out,
    void *k_cache, void *v_cache, const int32_t *block_table,
    int max_pages, int page_size, int num_pages,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/* Workspace bytes orthros_prefill_shard needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_prefill_shard_workspace_size(int B, int Tq, int Tkv, int Hq, int Hkv, int d,
                                                       int n_rows, int window, orthros_dtype dtype);

/*
 * One rank's share of a prefill whose token axis is cut into contiguous chunks
 * across devices (sequence parallelism: the paper runs its 64K-1M-token
 * prefills on 8 GPUs, Sec. 4.5 and the appendix's training/inference setup,
 * without describing the split). Eq. 4 needs only a halo of the w - 1 keys
 * before a chunk; Eq. 5 of an output row spans every chunk up to its position,
 * so each chunk contributes a normalised partial that orthros_merge_partials
 * combines exactly.
 *
 * The chunk holds Tq tokens at global positions P0 .. P0 + Tq - 1. Its keys
 * and values come with the H = Tkv - Tq tokens before it (the halo, received
 * from the ranks that own them; H >= min(w - 1, P0) makes the band rows exact):
 * k, v [B, Tkv, Hkv, d] hold positions P0 - H .. P0 + Tq - 1. Positions below
 * are in this buffer's coordinates (global position - P0 + H).
 *   - base rows (Eq. 4): q [B, Tq, Hq, d] are the chunk's raw queries; query
 *     i sits at position H + i and attends keys max(0, H + i - w + 1) .. H + i.
 *     o_base [B, Tq, Hq, d] (dtype), lse_base [B, Hq, Tq] float.
 *   - partial output rows (Eq. 5 over the chunk's own keys): row r of sequence b
 *     (row_indptr as out_indptr of orthros_prefill, HOST) at position t_r >= 0
 *     attends keys H .. min(t_r, Tkv - 1): rows owned by later ranks have
 *     t_r >= Tkv and read the whole chunk; a row with t_r < H reads nothing and
 *     gets o = 0, lse = -inf. q_rows [n_rows, Hq, d] are their raw
 *     output-stream queries (required when n_rows > 0).
 *     o_part [n_rows, Hq, d] float, lse_part [n_rows, Hq] float.
 * bf16 only (ORTHROS_EUNSUPPORTED otherwise); 1 <= Tq <= Tkv. A negative
 * row position sets ORTHROS_DEV_BAD_POSITION and that row is NaN. Workspace
 * and errors as for orthros_prefill.
 */
ORTHROS_API orthros_status orthros_prefill_shard(
    const void *q, const void *k, const void *v,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    const int32_t *row_indptr, const int32_t *row_positions, int n_rows,
    const void *q_rows,
    int B, int Tq, int Tkv, int Hq, int Hkv, int d, int window, float scale,
    orthros_dtype dtype,
    void *o_base, float *lse_base, float *o_part, float *lse_part,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/*
 * Exact merge of normalised attention partials of the same rows over disjoint
 * key sets: lse = log sum_p exp(lse_p), o = sum_p exp(lse_p - lse) o_p (each
 * set's share of the softmax denominator is exp(lse_p)). Merges the chunk
 * partials of orthros_prefill_shard into the rows of Eq. 5.
 * o_parts [n_parts, n_rows, Hq, d] float, lse_parts [n_parts, n_rows, Hq] float
 * o_out [n_rows, Hq, d] of element type dtype, lse_out [n_rows, Hq] float.
 * A partial with lse = -inf holds no keys and weighs nothing; a row whose
 * partials are all empty comes back empty (o = 0, lse = -inf), so partials
 * may be merged in any grouping. Needs no workspace.
 */
ORTHROS_API orthros_status orthros_merge_partials(const float *o_parts, const float *lse_parts, int n_parts,
                                                  int n_rows, int Hq, int d, orthros_dtype dtype,
                                                  void *o_out, float *lse_out, orthros_stream_t stream);

/* Workspace bytes orthros_prefill_backward needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_prefill_backward_workspace_size(int B, int T, int Hq, int Hkv, int d,
                                               int n_out, int window, orthros_dtype dtype);

/*
 * Backward of orthros_prefill for training in the pre-training and
 * fine-tuning regimes (Sec. 3.2): the gradients of a loss L with respect to
 * q, k, v, q_out and the four affine vectors, given dL/do of both streams.
 * The paper prints no backward; it is the chain rule through Eq. 4 and Eq. 5
 * (softmax attention) and through the affines q = alpha (.) q_raw + beta.
 * lse is an output the loss is taken not to depend on.
 *
 * Forward arguments (q .. scale, dtype) exactly as given to orthros_prefill,
 * except that out_positions must hold positions in [0, T) (repeats allowed).
 * o_base, lse_base, o_out, lse_out  the outputs orthros_prefill returned for
 *              them (o is used for D = dO . o, lse to recompute softmax weights)
 * do_base [B, T, Hq, d], do_out [n_out, Hq, d]: dL/do_base, dL/do_out
 * dq      [B, T, Hq, d]  dL/dq. When q_out is NULL the output rows read q at
 *              their positions, and their share is included here.
 * dk, dv  [B, T, Hkv, d] (both streams' shares)
 * dq_out  [n_out, Hq, d] dL/dq_out; required when q_out is given, else ignored
 * d_alpha_base, d_beta_base, d_alpha_out, d_beta_out [Hq, d] float
 * All gradients are overwritten (not accumulated into). Element tensors have
 * the dtype of q; lse and the affine gradients are float.
 * workspace    at least orthros_prefill_backward_workspace_size() bytes,
 *              256-byte aligned; contents on entry do not matter.
 * Errors as for orthros_prefill; an output position outside [0, T) sets
 * ORTHROS_DEV_BAD_POSITION and that row's dq_out (or share of dq) is NaN/absent.
 */
ORTHROS_API orthros_status orthros_prefill_backward(
    const void *q, const void *k, const void *v,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    const int32_t *out_indptr, const int32_t *out_positions, int n_out,
    const void *q_out,
    int B, int T, int Hq, int Hkv, int d, int window, float scale,
    orthros_dtype dtype,
    const void *o_base, const float *lse_base, const void *o_out, const float *lse_out,
    const void *do_base, const void *do_out,
    void *dq, void *dk, void *dv, void *dq_out,
    float *d_alpha_base, float *d_beta_base, float *d_alpha_out, float *d_beta_out,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/* Workspace bytes orthros_decode needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_decode_workspace_size(int B, int Hq, int Hkv, int d,
                                     int max_pages, int page_size,
                                     orthros_dtype dtype);

/*
 * One decoding step for B sequences (Sec. 3.2 "Decoding"; the decoupled
 * token pair of Sec. 3.1). For each sequence b with L = cache_lens[b]:
 *   1. the base token's K/V (k_new[b], v_new[b]) is written at position L of
 *      the paged cache (page block_table[b*max_pages + L/page_size], slot
 *      L % page_size);
 *   2. the base query (alpha/beta affine) attends keys max(0, L-w+1) .. L;
 *   3. the output query (alpha'/beta' affine) attends keys 0 .. L.
 * Both queries read the cache after the append.
 *
 * q            [B, Hq, d] raw query of the base token
 * q_out        [B, Hq, d] raw query of the output token, or NULL (= q)
 * k_new, v_new [B, Hkv, d]
 * k_cache, v_cache [num_pages, page_size, Hkv, d]  (modified: one slot per b)
 * block_table  [B, max_pages] int32 physical page ids
 * cache_lens   [B] int32 lengths BEFORE this step (read only; the caller
 *              increments them afterwards and provides a page for slot L)
 * o_base, o_out [B, Hq, d]; lse_base, lse_out [B, Hq] float
 * workspace    at least orthros_decode_workspace_size() bytes, 256-byte aligned
 */
ORTHROS_API orthros_status orthros_decode(
    const void *q, const void *q_out, const void *k_new, const void *v_new,
    void *k_cache, void *v_cache, const int32_t *block_table, int max_pages,
    int page_size, int num_pages, const int32_t *cache_lens,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    int B, int Hq, int Hkv, int d, int window, float scale, orthros_dtype dtype,
    void *o_base, float *lse_base, void *o_out, float *lse_out,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/* Workspace bytes orthros_extend needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_extend_workspace_size(int B, int n_new, int n_out, int Hq, int Hkv, int d,
                                     int max_pages, int page_size, orthros_dtype dtype);

/*
 * One continuous-batching step over the paged cache: a batch in which some
 * sequences append a prefill chunk, others decode one token, others nothing.
 * Sec. 3.2 runs every regime as the same computation (a prefill followed by
 * decoding steps agrees exactly with one longer prefill), so one call serves
 * them all; orthros_decode is the case of one new token per sequence.
 *
 * Sequence b (L = cache_lens[b]) appends its n_b = new_indptr[b+1] -
 * new_indptr[b] new tokens (rows new_indptr[b] .. of q, k_new, v_new) at
 * positions L .. L + n_b - 1 of its pages, then
 *   - every new token's base row attends keys max(0, t-w+1) .. t (Eq. 4);
 *   - every output row r (out_indptr[b] <= r < out_indptr[b+1]) at position
 *     out_positions[r] = t in [0, L + n_b) attends keys 0 .. t (Eq. 5), with
 *     raw query q_out[r], or, when q_out is NULL, the q of the new token at
 *     position t (t must then be a new position).
 *
 * q            [n_new, Hq, d] raw base queries of the new tokens
 * q_out        [n_out, Hq, d] raw output queries, or NULL (see above)
 * k_new, v_new [n_new, Hkv, d]
 * k_cache, v_cache [num_pages, page_size, Hkv, d] (modified: the appends)
 * block_table  [B, max_pages] int32; pages for positions < L + n_b must exist
 * cache_lens   [B] int32 device, lengths BEFORE the step (read only)
 * new_indptr, out_indptr  HOST [B+1] int32, start at 0, non-decreasing
 * out_positions [n_out] int32 device, absolute positions
 * o_base [n_new, Hq, d], lse_base [n_new, Hq], o_out [n_out, Hq, d],
 * lse_out [n_out, Hq] float
 * workspace    at least orthros_extend_workspace_size() bytes, 256-byte aligned
 * Rows whose data are impossible (a position outside its sequence, a length
 * past the block table) set ORTHROS_DEV_BAD_POSITION / _BAD_LENGTH and come
 * back as NaN; a page id outside [0, num_pages) sets ORTHROS_DEV_BAD_PAGE.
 */
ORTHROS_API orthros_status orthros_extend(
    const void *q, const void *q_out, const void *k_new, const void *v_new,
    void *k_cache, void *v_cache, const int32_t *block_table, int max_pages,
    int page_size, int num_pages, const int32_t *cache_lens,
    const int32_t *new_indptr, const int32_t *out_indptr, const int32_t *out_positions,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    int B, int Hq, int Hkv, int d, int window, float scale, orthros_dtype dtype,
    void *o_base, float *lse_base, void *o_out, float *lse_out,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/*
 * The shared Q/K/V projection that feeds the hot path (Alg. 1 lines 4-5,
 * Sec. 3.1): base-token rows x[0 .. n_base) and output-token rows
 * x[n_base .. n_base+n_out) are multiplied by ONE weight (in decoding, a
 * step's base and output tokens share its read), y = x W, and
 *   q_base = alpha_base (.) y_Q + beta_base   for base rows,
 *   q_out  = alpha_out  (.) y_Q + beta_out    for output rows,
 *   k, v   = y_K, y_V                         for base rows only (only the
 *            base stream writes the cache), to k_out / v_out and/or to the
 *            page slot of (token_seq[i], token_pos[i]).
 * The queries leave with their affine applied: pass identity affines
 * (alpha = 1, beta = 0) to the attention calls that read them.
 *
 * x        [n_base + n_out, d_model] bf16, d_model a multiple of 64
 * w_qkv    [(Hq + 2 Hkv) d, d_model] bf16: row j holds the weights of output
 *          column j (W transposed); columns are Q heads, then K, then V heads
 * alpha_*, beta_* [Hq, d] float
 * q_base [n_base, Hq, d], q_out [n_out, Hq, d] bf16 (q_out NULL if n_out = 0)
 * k_out, v_out [n_base, Hkv, d] bf16, or both NULL
 * k_cache, v_cache [num_pages, page_size, Hkv, d], block_table [B, max_pages],
 * token_seq, token_pos [n_base] device int32: all NULL for no cache writes
 * workspace at least 256 bytes (status word), 256-byte aligned
 * Errors: bf16 only (EUNSUPPORTED otherwise); a row whose page does not exist
 * sets ORTHROS_DEV_BAD_PAGE / _BAD_POSITION and its cache write is skipped.
 * The paper has no kernel for this step; it is the step upstream of the
 * attention that the decoding pair's shared weight read makes worth fusing.
 */
ORTHROS_API orthros_status orthros_qkv_project(
    const void *x, int n_base, int n_out, int d_model, const void *w_qkv,
    int Hq, int Hkv, int d,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    void *q_base, void *q_out, void *k_out, void *v_out,
    void *k_cache, void *v_cache, const int32_t *block_table, int B,
    int max_pages, int page_size, int num_pages,
    const int32_t *token_seq, const int32_t *token_pos, orthros_dtype dtype,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/*
 * orthros_decode without a workspace argument, for callers that cannot
 * allocate device memory where they run a decoding step (for example a host
 * framework whose operator interface passes only inputs and outputs, or a
 * serving loop whose allocator must not grow). The paper has no counterpart:
 * this is a deployment convenience, not part of the method.
 *
 * Same arguments, semantics and results as orthros_decode, minus workspace.
 * Scratch comes from one 32 MiB device array inside the library (held by
 * every GPU that loads it until the process exits); sizes whose
 * orthros_decode_workspace_size() exceeds that return ORTHROS_EWORKSPACE
 * before any launch. The first call on a device looks up the array's address
 * (cudaGetSymbolAddress) with that device current: make it before any stream
 * capture. All calls share the array: calls ordered on one stream are fine,
 * calls that overlap on the GPU race. Device-side status bits of this entry
 * point are not exposed; rows with bad data (or whose kernel gave up on a
 * bounded wait) come back as NaN. The array's address is kept per device for
 * the life of the process: resetting a device (cudaDeviceReset) after its
 * first call is not supported.
 */
ORTHROS_API orthros_status orthros_decode_static(
    const void *q, const void *q_out, const void *k_new, const void *v_new,
    void *k_cache, void *v_cache, const int32_t *block_table, int max_pages,
    int page_size, int num_pages, const int32_t *cache_lens,
    const float *alpha_base, const float *beta_base,
    const float *alpha_out, const float *beta_out,
    int B, int Hq, int Hkv, int d, int window, float scale, orthros_dtype dtype,
    void *o_base, float *lse_base, void *o_out, float *lse_out,
    orthros_stream_t stream);

/*
 * Rotary positions. The pages leave the positional encoding of the converted
 * models aside (Alg. 1 projects, applies the stream's affine and attends);
 * models with rotary positions turn each query and key between those two
 * steps. Pair i of a head at position t turns by the angle t * freq[i]:
 *   (y_a, y_b) = amplitude * (u_a cos - u_b sin, u_a sin + u_b cos),
 * over the first rot_dim channels of the head, paired (i, i + rot_dim/2) in
 * the half layout or (2i, 2i + 1) in the interleaved one; channels past
 * rot_dim keep u. The attention calls then take identity affines.
 */
typedef enum { ORTHROS_ROPE_HALF = 0, ORTHROS_ROPE_INTERLEAVED = 1 } orthros_rope_layout;

/*
 * How orthros_rotary_frequencies scales the plain frequencies
 * f_i = base^(-2i/rot_dim) for contexts `factor` times the original_length a
 * model was trained on:
 *   PLAIN    f_i
 *   LINEAR   f_i / factor (position interpolation)
 *   STRETCH  base * factor^(rot_dim/(rot_dim-2)) in place of base (the
 *            "NTK-aware" rule: the highest frequency kept, the lowest divided
 *            by factor)
 *   BANDS    by the turns r = original_length * f_i / 2 pi that a frequency
 *            makes over the original length: f_i / factor below low_turns, f_i
 *            above high_turns, ((1-s) / factor + s) f_i between, with
 *            s = (r - low_turns) / (high_turns - low_turns)
 *   BANDS_TEMPERED  BANDS with amplitude 0.1 ln(factor) + 1 on cos and sin
 *            (YaRN, published with low_turns 1 and high_turns 32; BANDS is common
 *            with 1 and 4; the other rules have amplitude 1)
 */
typedef enum {
    ORTHROS_ROPE_PLAIN = 0,
    ORTHROS_ROPE_LINEAR = 1,
    ORTHROS_ROPE_STRETCH = 2,
    ORTHROS_ROPE_BANDS = 3,
    ORTHROS_ROPE_BANDS_TEMPERED = 4
} orthros_rope_scaling;

/*
 * freq HOST [rot_dim/2] double (radians per position) and *amplitude HOST of
 * a scaling rule. rot_dim even and >= 2 (>= 4 for STRETCH), base > 1, factor
 * >= 1 (1 for PLAIN is customary; it is not read there); original_length > 0
 * and 0 <= low_turns < high_turns for the two BANDS rules (not read by the
 * others).
 */
ORTHROS_API orthros_status orthros_rotary_frequencies(int rot_dim, double base, orthros_rope_scaling rule, double factor,
                                                      double original_length, double low_turns, double high_turns,
                                                      double *freq, float *amplitude);

/*
 * freq HOST [n] (radians per position, finite) -> steps HOST [n]: the fraction
 * of a turn per position in units of 2^-64, rounded to the nearest. The calls
 * below take a device copy of steps: position times step, modulo 2^64, is the
 * phase at any 32-bit position to 2^-34 turn, where a float product has lost its
 * fraction.
 */
ORTHROS_API orthros_status orthros_rotary_steps(const double *freq, int n, uint64_t *steps);

/*
 * Rotates n tokens: y = amplitude R(t) u with u = alpha (.) x + beta.
 *
 * x, y         [n, H, d]: token i starts x_stride (y_stride) elements after
 *              token i - 1; the heads of a token are contiguous. Strides are
 *              multiples of 16 bytes; y_stride >= H d. So slices of a packed
 *              projection need no copy. y may be x (same stride); the
 *              elements of x and y must not overlap otherwise.
 * positions    [n] int32, any value
 * alpha, beta  [H, d] float (16-byte aligned), or both NULL (u = x)
 * steps        [rot_dim/2] device copy of orthros_rotary_steps' output
 * rot_dim      a multiple of 16, 16 <= rot_dim <= d
 * Computed in fp32 and rounded once to dtype. No workspace, no status word.
 */
ORTHROS_API orthros_status orthros_rotate(const void *x, long long x_stride, const int32_t *positions,
                                          const float *alpha, const float *beta, const uint64_t *steps, int rot_dim,
                                          orthros_rope_layout layout, float amplitude, int n, int H, int d,
                                          orthros_dtype dtype, void *y, long long y_stride, orthros_stream_t stream);

/* Workspace bytes orthros_rotate_backward needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_rotate_backward_workspace_size(int n, int H, int d, orthros_dtype dtype);

/*
 * Gradients of orthros_rotate: with g = amplitude R(-t) dy (g = dy past
 * rot_dim), dx = alpha (.) g, d_alpha = sum over tokens of g (.) x, d_beta =
 * sum over tokens of g.
 *
 * dy, dx       [n, H, d] with strides as for orthros_rotate; dx may be dy
 * x, x_stride  the forward's input; read only for d_alpha
 * alpha        [H, d] float, or NULL (1)
 * d_alpha, d_beta [H, d] float, overwritten, or both NULL (then x and the
 *              workspace are not read and may be NULL). The sums run in a fixed
 *              order: the same call gives the same bits.
 * workspace    at least orthros_rotate_backward_workspace_size() bytes,
 *              256-byte aligned; contents on entry do not matter.
 */
ORTHROS_API orthros_status orthros_rotate_backward(const void *dy, long long dy_stride, const void *x,
                                                   long long x_stride, const int32_t *positions, const float *alpha,
                                                   const uint64_t *steps, int rot_dim, orthros_rope_layout layout,
                                                   float amplitude, int n, int H, int d, orthros_dtype dtype, void *dx,
                                                   long long dx_stride, float *d_alpha, float *d_beta,
                                                   void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/*
 * Appends new tokens to the paged cache with the rotation applied on the way,
 * and rotates both query streams in the same call.
 *   - new token i (sequence token_seq[i], position token_pos[i]): its key
 *     heads are rotated and written to its page slot (page
 *     block_table[seq*max_pages + pos/page_size], slot pos % page_size), its
 *     values are copied there;
 *   - q_rot[i] = R(token_pos[i]) (alpha_base (.) q[i] + beta_base) (skipped
 *     when q is NULL);
 *   - q_out_rot[r] = R(out_positions[r]) (alpha_out (.) q_out[r] + beta_out)
 *     for the n_out output-stream rows.
 *
 * q [n_new, Hq, d], q_out [n_out, Hq, d], k_new, v_new [n_new, Hkv, d], each
 *              with its token stride in elements (a multiple of 16 bytes), as
 *              slices of a packed projection have them
 * alpha_*, beta_* [Hq, d] float, each pair both set or both NULL (identity; as
 *              after orthros_qkv_project, which applies the affines itself)
 * token_seq, token_pos [n_new], out_positions [n_out] device int32. No two
 *              new tokens may share a slot.
 * steps, rot_dim, layout, amplitude as for orthros_rotate
 * q_rot [n_new, Hq, d], q_out_rot [n_out, Hq, d], contiguous
 * k_cache, v_cache [num_pages, page_size, Hkv, d], block_table [B, max_pages]
 * workspace    at least 256 bytes (status word), 256-byte aligned
 * A sequence outside [0, B) or a position outside its block table sets
 * ORTHROS_DEV_BAD_POSITION, a page id outside [0, num_pages)
 * ORTHROS_DEV_BAD_PAGE; that token's cache write is skipped.
 */
ORTHROS_API orthros_status orthros_rotate_append(
    const void *q, long long q_stride, const void *q_out, long long q_out_stride, const void *k_new, long long k_stride,
    const void *v_new, long long v_stride, const float *alpha_base, const float *beta_base, const float *alpha_out,
    const float *beta_out, const uint64_t *steps, int rot_dim, orthros_rope_layout layout, float amplitude,
    const int32_t *token_seq, const int32_t *token_pos, const int32_t *out_positions, int n_new, int n_out, int Hq,
    int Hkv, int d, orthros_dtype dtype, void *q_rot, void *q_out_rot, void *k_cache, void *v_cache,
    const int32_t *block_table, int B, int max_pages, int page_size, int num_pages, void *workspace,
    size_t workspace_bytes, orthros_stream_t stream);

/* Workspace bytes orthros_chunk_attention needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_chunk_attention_workspace_size(int B, int n, int max_new, int Hq, int Hkv, int d,
                                                          int max_pages, int page_size, orthros_dtype dtype);

/*
 * Attention of new tokens over a paged cache that already holds their keys
 * and values (orthros_rotate_append or orthros_qkv_project wrote them): one
 * query stream of a serving step, any mix of single tokens (decoding) and
 * chunks of a prompt. Sequence b's n_b = q_indptr[b+1] - q_indptr[b] tokens
 * are the last n_b of its kv_lens[b] cached ones: token i sits at position
 * t = kv_lens[b] - n_b + i and attends keys max(0, t-w+1) .. t. With the
 * window of the base stream this is Eq. 4; with window >= kv_lens it is Eq. 5,
 * the output stream's row (its last token alone, or a whole chunk).
 *
 * q            [n, Hq, d] bf16, used as they are (affine and rotation applied
 *              before)
 * q_indptr     [B+1] int32 DEVICE, 0 .. n, non-decreasing
 * kv_lens      [B] int32 DEVICE: cached tokens, the new ones included
 * max_new      upper bound of the n_b (sizes the workspace; n always serves). The
 *              order in which the parts of a row are joined goes by it: the same
 *              call gives the same bits, one with another bound may round otherwise
 * k_cache, v_cache [num_pages, page_size, Hkv, d], block_table [B, max_pages]
 *              DEVICE int32; any page_size (multiples of 8 are copied by TMA,
 *              others row by row, slower)
 * o [n, Hq, d] bf16, lse [n, Hq] float or NULL
 * scale        > 0
 * workspace    at least orthros_chunk_attention_workspace_size() bytes,
 *              256-byte aligned; contents on entry do not matter.
 * Every length is read on the device: a step can be captured once and replayed
 * while the lengths grow. bf16 only; at most 128 query heads per kv head.
 * Keys and values that any row of the call sees must be finite (one that is not
 * may also make NaN rows of its sequence that do not see it); what pages hold
 * past a sequence's length, or before every window of the call, does not matter.
 * Products accumulate in fp32, as do the running maximum, the sum and o; softmax
 * weights are rounded to bf16 for their product with v, as in the other bf16
 * calls: half a step, 2^-8, of each term.
 * A q_indptr that does not run from 0 to n sets ORTHROS_DEV_BAD_LENGTH and
 * every row is NaN; n_b > max_new, kv_lens[b] < n_b or past the block table
 * sets it for that sequence's rows. A page id outside [0, num_pages) sets
 * ORTHROS_DEV_BAD_PAGE and the rows that see its keys are NaN (as are those that
 * see only keys between two such pages closer than 128 tokens). A row whose
 * logits are all -inf (an infinite query) has no softmax: o is NaN, lse -inf.
 */
ORTHROS_API orthros_status orthros_chunk_attention(const void *q, const int32_t *q_indptr, const int32_t *kv_lens,
                                                   const void *k_cache, const void *v_cache,
                                                   const int32_t *block_table, int B, int n, int max_new, int Hq,
                                                   int Hkv, int d, int window, float scale, orthros_dtype dtype,
                                                   int max_pages, int page_size, int num_pages, void *o, float *lse,
                                                   void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/*
 * orthros_rotate with a norm of each head before the affine (models that norm
 * queries and keys): y = amplitude R(t) u with
 *   u = alpha (.) (weight (.) xh) + beta,  xh = x / sqrt(mean_c x_c^2 + eps),
 * the mean over the d channels of the head.
 *
 * weight       [d] float (16-byte aligned), shared by the heads, or NULL (1)
 * eps          > 0
 * The other arguments are orthros_rotate's. The squares are summed in fp32: a
 * head whose sum of squares is past 3.4e38 has xh = 0.
 */
ORTHROS_API orthros_status orthros_norm_rotate(const void *x, long long x_stride, const int32_t *positions,
                                               const float *weight, float eps, const float *alpha, const float *beta,
                                               const uint64_t *steps, int rot_dim, orthros_rope_layout layout,
                                               float amplitude, int n, int H, int d, orthros_dtype dtype, void *y,
                                               long long y_stride, orthros_stream_t stream);

/* Workspace bytes orthros_norm_rotate_backward needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_norm_rotate_backward_workspace_size(int n, int H, int d, orthros_dtype dtype);

/*
 * Gradients of orthros_norm_rotate: with g = amplitude R(-t) dy, r = 1 /
 * sqrt(mean x^2 + eps), a = alpha (.) weight and S = sum over tokens of
 * g (.) xh (per head),
 *   dx = r (a (.) g - xh mean_c(a g xh)),   d_beta = sum over tokens of g,
 *   d_alpha = weight (.) S,                 d_weight = sum over heads of alpha (.) S.
 *
 * d_weight     [d] float, overwritten, or NULL
 * d_alpha, d_beta [H, d] float, overwritten, or both NULL
 * x            the forward's input, always read
 * The other arguments are orthros_rotate_backward's (dx may be dy; without
 * gradients of weight and affine the workspace may be NULL). The sums run in a
 * fixed order: the same call gives the same bits. A head with xh = 0 for its size
 * (orthros_norm_rotate) has r = 0, and so dx = 0.
 */
ORTHROS_API orthros_status orthros_norm_rotate_backward(
    const void *dy, long long dy_stride, const void *x, long long x_stride, const int32_t *positions, const float *weight,
    float eps, const float *alpha, const uint64_t *steps, int rot_dim, orthros_rope_layout layout, float amplitude, int n, int H,
    int d, orthros_dtype dtype, void *dx, long long dx_stride, float *d_weight, float *d_alpha, float *d_beta,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/*
 * orthros_rotate_append with norms, and with the place of a new token in the
 * cache given apart from its position (the tokens of a drafted tree lie one
 * behind the other, while their positions are their depths):
 *   - key i is normed with k_weight, rotated to token_pos[i] and written to
 *     token slot token_slots[i] (page * page_size + place in the page), its
 *     values copied there;
 *   - q_rot[i] and q_out_rot[r] as orthros_norm_rotate gives them for q[i] at
 *     token_pos[i] and q_out[r] at out_positions[r], with q_weight and the
 *     stream's affine.
 *
 * token_slots  [n_new] int32, as orthros_plan_step makes them; -1: the token is
 *              not cached (a row of padding). No two tokens may share a slot.
 * q_weight, k_weight [d] float (16-byte aligned) or NULL (1)
 * eps          > 0, or 0 for no norm (both weights NULL): slots alone
 * The other arguments are orthros_rotate_append's. A slot below -1 or past the
 * pool sets ORTHROS_DEV_BAD_PAGE; that token's cache write is skipped.
 */
ORTHROS_API orthros_status orthros_norm_rotate_append(
    const void *q, long long q_stride, const void *q_out, long long q_out_stride, const void *k_new, long long k_stride,
    const void *v_new, long long v_stride, const float *q_weight, const float *k_weight, float eps, const float *alpha_base,
    const float *beta_base, const float *alpha_out, const float *beta_out, const uint64_t *steps, int rot_dim,
    orthros_rope_layout layout, float amplitude, const int32_t *token_slots, const int32_t *token_pos,
    const int32_t *out_positions, int n_new, int n_out, int Hq, int Hkv, int d, orthros_dtype dtype, void *q_rot,
    void *q_out_rot, void *k_cache, void *v_cache, int page_size, int num_pages, void *workspace, size_t workspace_bytes,
    orthros_stream_t stream);

/*
 * What a serving step needs from its lengths, made on the GPU. Sequence b has
 * cache_lens[b] tokens in the cache and new_lens[b] new ones; it needs
 * ceil((cache + new) / page_size) pages and takes those that it does not hold
 * yet from the free pages.
 *
 * cache_lens, new_lens, pages_held [B] int32; new_lens[b] = -1: the sequence has
 *              ended, all its pages go back (cache_lens is then not read further)
 * free_pages   [num_pages], free_count [1]: the first free_count entries are the
 *              free pages, a stack, updated in place. Ended sequences push theirs,
 *              in order, first; then the growing sequences, in order, take from the
 *              top. (A later one does not get what an earlier one found too little
 *              of.) Entries from the new height on mean nothing.
 * block_table  [B, max_pages]: entries of new pages are written, others left
 * n            rows of the token arrays; rows behind the last new token are
 *              padding: token_seq -1, token_pos 0, token_slots -1, no mask bits
 *              (rows to spare are for orthros_tree_attention; consecutive tokens whose
 *              number varies, up to 256 a sequence, are trees in which every token's
 *              parent is the one before it)
 * parents      [n] with max_tree > 0 (at most 256): the new tokens of every
 *              sequence are a drafted tree of at most max_tree tokens, and
 *              parents[i] is the number within its tree (0, 1, ...) of token i's
 *              parent, which comes before it, or -1 under the last cached token.
 *              NULL with max_tree = 0: consecutive tokens
 * q_indptr [B+1], token_seq, token_pos, token_slots [n], kv_lens [B] (cache + new;
 *              0 once ended; -1 without a place in the step): as
 *              orthros_norm_rotate_append, orthros_chunk_attention (for which n has
 *              to be the number of tokens) and orthros_tree_attention take them.
 *              Token j of sequence b lies at place cache_lens[b] + j; its position
 *              is that place, or in a tree cache_lens[b] + its depth.
 * tree_mask    [n, ceil(max_tree / 32)]: bit j of word j/32 of token i's row is
 *              set for token j of its tree if that is i or one of i's ancestors
 * cache_lens_out [B] or NULL, pages_held_out [B], free_count_out [1]: the state
 *              after the step, all new tokens counted (orthros_tree_commit sets the
 *              lengths after a tree's verification). They may be cache_lens,
 *              pages_held and free_count; outputs must not overlap inputs otherwise.
 * workspace    at least 256 bytes (status word), 256-byte aligned. B <= 8192.
 * A sequence whose lengths cannot be (negative, past the block table, a tree
 * over max_tree) sets ORTHROS_DEV_BAD_LENGTH, one whose pages are not all there
 * ORTHROS_DEV_NO_PAGES: it has no place in the step. Nothing of its state changes,
 * and its token rows are padding, which the attention makes NaN. More tokens than
 * rows, or a stack that cannot hold the pages, set ORTHROS_DEV_BAD_LENGTH and
 * refuse the step: no state changes, q_indptr and kv_lens are all -1. A page id outside
 * [0, num_pages) sets ORTHROS_DEV_BAD_PAGE where the step meets it: under a new token
 * (slot -1), among the pages taken from the stack (the table has it), or among those of
 * an ended sequence, which then has not ended: nothing of its state changes, its kv_lens
 * is -1 and none of its pages goes back. (Pages that hold only older tokens are not
 * looked up here.) A parent that does not come before its token sets
 * ORTHROS_DEV_BAD_POSITION (counted as -1).
 */
ORTHROS_API orthros_status orthros_plan_step(
    const int32_t *cache_lens, const int32_t *new_lens, const int32_t *pages_held, const int32_t *free_count,
    const int32_t *parents, int max_tree, int32_t *free_pages, int32_t *block_table, int B, int n, int max_pages, int page_size,
    int num_pages, int32_t *q_indptr, int32_t *kv_lens, int32_t *cache_lens_out, int32_t *pages_held_out, int32_t *free_count_out,
    int32_t *token_seq, int32_t *token_pos, int32_t *token_slots, int32_t *tree_mask, void *workspace, size_t workspace_bytes,
    orthros_stream_t stream);

/* Workspace bytes orthros_tree_attention needs for these sizes (0 if rejected). */
ORTHROS_API size_t orthros_tree_attention_workspace_size(int B, int n, int max_new, int Hq, int Hkv, int d, int max_pages,
                                                         int page_size, orthros_dtype dtype);

/*
 * Attention of drafted trees over a paged cache that already holds their keys
 * and values: orthros_chunk_attention with a mask over the new tokens. The n_b =
 * q_indptr[b+1] - q_indptr[b] tokens of sequence b lie at places L .. L + n_b - 1,
 * L = kv_lens[b] - n_b. Token i sees token j of its own tree where bit j of its
 * mask row is set; its position is t_i = L + max(bits, 1) - 1, bits being the
 * number of tokens that it sees. It sees the keys before the tree from
 * max(0, t_i - w + 1) on, and of the tree those at positions above t_i - w.
 *
 * q_indptr     [B+1] int32 DEVICE, from 0, non-decreasing, to at most n: rows
 *              behind q_indptr[B] are left as they were
 * tree_mask    [n, mask_words] int32, mask_words in [1, 8]; bits of tokens that
 *              the tree does not have count for nothing. Any mask will do, also
 *              one with later tokens or without the token itself: a row that sees
 *              no key at all has o = 0, lse = -inf
 * max_new      upper bound of the n_b (32 mask_words always serves)
 * The other arguments, the precision and the reports are orthros_chunk_attention's.
 * The keys and values of all n_b tokens, and the cached ones from max(0, L - w + 1)
 * on, must be finite.
 */
ORTHROS_API orthros_status orthros_tree_attention(
    const void *q, const int32_t *q_indptr, const int32_t *kv_lens, const int32_t *tree_mask, int mask_words,
    const void *k_cache, const void *v_cache, const int32_t *block_table, int B, int n, int max_new, int Hq, int Hkv, int d,
    int window, float scale, orthros_dtype dtype, int max_pages, int page_size, int num_pages, void *o, float *lse,
    void *workspace, size_t workspace_bytes, orthros_stream_t stream);

/*
 * After a tree's verification: the accepted path's keys and values move from
 * places L + accepted[b][i] to L + i, so that the cache holds consecutive tokens
 * again, and cache_lens[b] = L + n_accepted[b].
 *
 * k_cache, v_cache [layers, num_pages, page_size, Hkv, d]: all layers at once
 * q_indptr, kv_lens, block_table: the tree step's
 * accepted     [B, most] int32, ascending tokens of the tree (numbers within it);
 *              the first n_accepted[b] of a row count. most in [1, 256]
 * cache_lens   [B], written; not kv_lens
 * Sequences own the pages of their trees. Places behind L + n_accepted keep what
 * they had. workspace: at least 256 bytes (status word), 256-byte aligned.
 * A path that does not ascend or leaves the tree sets ORTHROS_DEV_BAD_POSITION,
 * n_accepted outside [0, min(most, n_b)] ORTHROS_DEV_BAD_LENGTH, a page id outside
 * [0, num_pages) ORTHROS_DEV_BAD_PAGE: nothing of that sequence moves, and
 * cache_lens[b] = L. Impossible lengths (n_b < 0, kv_lens[b] < n_b, as of a sequence
 * that had no place in the plan, or past the block table) set ORTHROS_DEV_BAD_LENGTH
 * and leave cache_lens[b] as it was.
 */
ORTHROS_API orthros_status orthros_tree_commit(void *k_cache, void *v_cache, int layers, const int32_t *block_table,
                                               const int32_t *q_indptr, const int32_t *kv_lens, const int32_t *accepted,
                                               const int32_t *n_accepted, int most, int B, int Hkv, int d,
                                               orthros_dtype dtype, int max_pages, int page_size, int num_pages,
                                               int32_t *cache_lens, void *workspace, size_t workspace_bytes,
                                               orthros_stream_t stream);

/*
 * Synchronises `stream`, reads the status word that the last call using
 * `workspace` left there and returns ORTHROS_OK, ORTHROS_EDEVICE (data bits) or
 * ORTHROS_ETIMEOUT (timeout bit). *bits (if not NULL) receives the raw
 * ORTHROS_DEV_* bits. This is the one call that blocks the host.
 */
ORTHROS_API orthros_status orthros_check(const void *workspace, orthros_stream_t stream,
                             uint32_t *bits);

/*
 * Per-kernel timing of the library's own launches (tracing aid).
 * orthros_profile_begin() starts recording: every kernel the library launches
 * afterwards is bracketed by two CUDA events recorded on its launch stream.
 * orthros_profile_end() stops recording, waits for the recorded events and
 * fills up to max_entries records, one per kernel name, in first-launch order.
 * It returns the number of distinct kernels (may exceed max_entries), or -1 on
 * a CUDA error. Recording is process-wide and not thread-safe; it adds two
 * event records per launch and nothing else.
 */
typedef struct {
    char name[48];   /* kernel family, e.g. "prefill_tc" */
    int launches;    /* launches recorded */
    double total_ms; /* summed event-to-event time of those launches */
} orthros_kernel_time;

ORTHROS_API orthros_status orthros_profile_begin(void);
ORTHROS_API int orthros_profile_end(orthros_kernel_time *out, int max_entries);

/*
 * Self-test of the failure path (no counterpart in the paper): launches one
 * small kernel whose only wait is on an mbarrier that nothing arrives on,
 * bounded by limit_cycles SM clock cycles (1 .. about 4e9). The wait runs out,
 * the kernel raises ORTHROS_DEV_TIMEOUT in the workspace's status word and
 * returns; orthros_check(workspace, ...) then reports ORTHROS_ETIMEOUT. Every
 * kernel of the library that waits on a barrier uses the same bounded wait
 * (with a limit of about 2 s), so a stalled pipeline ends with this status
 * instead of a hang. workspace: at least 256 bytes, 256-byte aligned.
 */
ORTHROS_API orthros_status orthros_selftest_wait_timeout(long long limit_cycles, void *workspace,
                                                         size_t workspace_bytes, orthros_stream_t stream);

/* Static English name of a status code. */
ORTHROS_API const char *orthros_status_string(orthros_status s);

/* Description of the last host-side error on this thread ("" if none). */
ORTHROS_API const char *orthros_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ORTHROS_ATTN_H */
