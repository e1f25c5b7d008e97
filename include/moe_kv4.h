/*
 * moe_kv4.h -- C ABI of the 4-bit paged key/value cache and its attention for one
 * NVIDIA GB300 (sm_103a): the attention half of the decoder layer whose expert
 * MLP is in moe_int4.h.  The conventions of that header hold (device pointers of
 * the caller, stream-ordered asynchronous calls, bf16 as bit patterns, MOE_OK or a
 * negative MOE_ERR_* code, no allocation); the entry points live in the same
 * library and moe_int4_strerror names their codes.
 *
 * Values.  Keys and values are held like the INT4 expert weights: a code q in
 * 0..15 and one scale for 32 consecutive dimensions of one token and head,
 * value = (q - 8) * scale.  The scale is a bf16 number in [2^-14, 2720], stored
 * as fp16 (exact), so every value is exact in fp16.  Quantisation of x[0..31]:
 *   scale = clamp(bf16(max|x| * fp32(1/7)), 2^-14, 2720)
 *   q     = clamp(rint(x / scale), -8, 7) + 8        (fp32, nearest even)
 *
 * Layout.  pages is [layers][n_pages][kv_heads][block], one block the tokens of
 * one page and head: with P = page_size, D = head_dim, NG = D / 32,
 *   K codes [P][D/2] | V codes [P][D/2] | K scales fp16 [P][NG] | V scales [P][NG]
 * (moe_kv4_block_bytes = P * (D + D/8) bytes).
 *   K row: 32-bit word t*NG + G (t = 0..3, G = 0..NG-1) holds dimension
 *          32G + 8t + 2i + h at bits 16h + 4i (i = 0..3, h = 0, 1).
 *   V row: 16-bit piece g*NG + G (g = 0..7) holds dimension 32G + 4g + i at bits 4i.
 * A lane of a tensor-core instruction finds the eight K dimensions (four V
 * dimensions of each group) that it multiplies in one word, in operand order.
 *
 * Sequences.  Token j of sequence b lies in slot j % P of page
 * tables[b][j / P].  Only slots below a sequence's length are read as numbers: what
 * unused slots hold (anything, NaN scales included) never reaches a result.
 *
 * Device-side faults of the data set a bit and count in the error words
 * (uint32[2]: flags, count), as in moe_int4.h: nothing traps.
 */
#ifndef MOE_KV4_H
#define MOE_KV4_H

#include "moe_int4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_KV4_DEVERR_PAGE 0x10u      /* a page id outside [0, n_pages) that a token needs, or a
                                          length beyond its table: those tokens are skipped */
#define MOE_KV4_DEVERR_POSITION 0x20u  /* a rotary position outside [0, max_pos): the nearest
                                          one is used */
#define MOE_KV4_DEVERR_RANGE 0x40u     /* a key or value beyond +-19040 or not finite was
                                          saturated (NaN: 0), or a query beyond +-65504 or not
                                          finite was saturated */
#define MOE_KV4_DEVERR_NO_PAGES 0x80u  /* the pool had too few free pages: the request, and those
                                          after it in the call, were left as they were */
#define MOE_KV4_DEVERR_SEQ 0x100u      /* a sequence id out of range, a fork into a sequence that
                                          holds tokens, a length that shrinks, or a page freed
                                          more often than it was taken: that request is skipped */

/* The pool.  1 <= layers <= 1024, 1 <= n_pages <= 1<<20, 1 <= kv_heads <= 256,
 * head_dim 64 or 128, page_size 16, 32 or 64. */
typedef struct {
    int32_t layers;
    int32_t n_pages;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t page_size;
} moe_kv4_shape;

/* A batch of requests: request b has new tokens cu_q[b]..cu_q[b+1]-1 of the call
 * (any number, zero included), which are the last ones of its kv_len[b] tokens.
 * A request with more new tokens than kv_len is a contract violation whose
 * surplus first tokens see nothing and are not stored.  A request whose rows are not
 * 0 <= cu_q[b] <= cu_q[b+1] <= tokens is left out.  tokens may exceed
 * cu_q[requests] (a batch padded to a captured step's size): rows of the call that no
 * request owns are not stored, read as 0 and get no attention output. */
typedef struct {
    int32_t requests;       /* 0..65536 */
    int32_t tokens;         /* rows of q, k, v and the outputs, cu_q[requests] of them in use;
                               0..1<<20 */
    int32_t max_q;          /* largest number of new tokens of a request (an upper bound) */
    int32_t max_kv;         /* largest kv_len (an upper bound) */
    int32_t table_stride;   /* entries from one row of tables to the next (its capacity) */
    const int32_t *cu_q;    /* [requests + 1] */
    const int32_t *kv_len;  /* [requests]; attention cuts lengths at 2^31 - 2^22 */
    const int32_t *tables;  /* [requests][table_stride] */
} moe_kv4_batch;

/* Sequences that page management works on. */
typedef struct {
    int32_t seqs;          /* rows of tables, entries of lens; 1..65536 */
    int32_t table_stride;  /* entries per row */
    int32_t *tables;       /* [seqs][table_stride]; entries past a sequence's pages are -1 */
    int32_t *lens;         /* [seqs] tokens */
    int32_t *refs;         /* [n_pages] how many tables hold the page (0: free) */
} moe_kv4_seqs;

/* Bytes of one block (one page of one head) and of the whole pool; 0 for an
 * unsupported shape. */
size_t moe_kv4_block_bytes(const moe_kv4_shape *shape);
size_t moe_kv4_pool_bytes(const moe_kv4_shape *shape);

/*
 * moe_kv4_append: the head norms, the position rotation and the cache write of a
 * batch's new tokens, in one pass.
 *   y = x / sqrt(mean(x^2) + eps) * weight     over each head of q and of k
 *   (a, b) -> (a cos - b sin, b cos + a sin)   for its D/2 pairs of dimensions
 * In:  q, k, v    bf16, heads of D contiguous values, heads of a token contiguous;
 *                 *_stride elements from one token to the next (a multiple of 8),
 *                 so that all three may be parts of one projection's output.
 *                 q may be NULL (nothing is written to q_out).
 *      q_weight, k_weight  bf16 [D]; NULL: no norm.
 *      cos, sin   fp32 [max_pos][D/2]; both NULL: no rotation.  The row is
 *                 positions[t] (int32 [tokens]; NULL: the token's index in its
 *                 sequence).  interleaved 0: pairs (i, i + D/2); 1: (2i, 2i + 1).
 * Out: q_out      bf16 [tokens][q_heads][D] contiguous; may be q itself when q is
 *                 contiguous, else must not overlap the inputs.
 *      pages      the tokens' slots of layer `layer`: k after norm and rotation, v.
 * Everything is fp32 with each operation rounded on its own, in a fixed order, so
 * results are reproducible bit for bit: squares are added as
 * s[j] = x[j]^2 + x[j + D/2]^2, each run of eight of them as
 * ((s0+s4)+(s2+s6)) + ((s1+s5)+(s3+s7)), and the D/16 runs pairwise; then
 * x * (1 / sqrt(sum * (1/D) + eps)) * weight.
 * err: uint32[2] or NULL.  Errors: MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_ALIGN,
 *   MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA.
 */
int moe_kv4_append(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                   const uint16_t *v, int64_t v_stride, const uint16_t *q_weight,
                   const uint16_t *k_weight, float eps, const float *cos, const float *sin,
                   const int32_t *positions, int max_pos, int interleaved, int q_heads,
                   uint16_t *q_out, void *pages, int layer, const moe_kv4_shape *shape,
                   const moe_kv4_batch *batch, uint32_t *err, moe_stream_t stream);

/* moe_kv4_read: the batch's new tokens as the cache holds them, dequantised:
 * k_out, v_out fp16 [tokens][kv_heads][D] (either may be NULL).  Tokens without a
 * valid page read as 0.  (With cu_q the running sum of kv_len it reads whole
 * sequences.)  Errors as moe_kv4_append. */
int moe_kv4_read(const void *pages, int layer, const moe_kv4_shape *shape,
                 const moe_kv4_batch *batch, uint16_t *k_out, uint16_t *v_out, uint32_t *err,
                 moe_stream_t stream);

/* Workspace bytes of moe_kv4_attention for this pool shape and number of query
 * heads, for any batch. */
size_t moe_kv4_workspace_bytes(const moe_kv4_shape *shape, int q_heads);

/*
 * moe_kv4_attention: out[t, h] = sum_j softmax_j(scale * q[t,h] . k[j]) v[j] over
 * the tokens j of t's sequence that t sees, with kv head h / (q_heads / kv_heads).
 * With p = t's index in its sequence, t sees j <= p; of these
 *   window > 0: only j > p - window (0: all); pages wholly before every row's window
 *     are not read, and their table entries may be anything;
 *   tree (uint64 [tokens], NULL: none): of the request's new tokens only those
 *     whose bit is set, bit i for its i-th new token (requests of at most 64 new
 *     tokens): a tree of drafts, each seeing its ancestors and itself.
 * A row that sees nothing gives zeros and lse -inf.
 * In:  q          bf16, q_stride elements from token to token (a multiple of 8).
 *      q_heads    a multiple of kv_heads, up to 64 for each kv head.
 * Out: out        bf16 [tokens][q_heads][D].
 *      lse        fp32 [tokens][q_heads], natural log of the sum of exponentials;
 *                 NULL: not written.
 * workspace: >= moe_kv4_workspace_bytes, 16-byte aligned; its first
 *   MOE_KV4_WS_HEADER bytes are zeroed once when it is allocated (the first two
 *   words are the error words, which accumulate; the rest returns to zero after
 *   every call, but for one that reports MOE_DEVERR_TIMEOUT: zero it again).  Calls
 *   in flight at once must not share it.
 * The softmax statistics, scores and sums are fp32; q is converted to fp16 (exact
 * for magnitudes in [2^-14, 65504], in steps of 2^-24 below) and the unnormalised
 * probabilities to fp16 (11 significant bits down to 2^-21 of the row's maximum, steps
 * of 2^-31 below) for the tensor cores.  How a sequence is split over the GPU depends on
 * the batch; for equal arguments results are equal bit for bit.
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE,
 *   MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA.
 */
#define MOE_KV4_WS_HEADER 8192
int moe_kv4_attention(const uint16_t *q, int64_t q_stride, int q_heads, const void *pages,
                      int layer, const moe_kv4_shape *shape, const moe_kv4_batch *batch,
                      float scale, int window, const uint64_t *tree, uint16_t *out, float *lse,
                      void *workspace, size_t workspace_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Pages                                                                      */
/* ------------------------------------------------------------------------- */

/* Scratch bytes (device, 16-byte aligned, no initial contents) that the calls
 * below need for n requests. */
size_t moe_kv4_scratch_bytes(const moe_kv4_shape *shape, int n);

/* moe_kv4_reserve: sequence ids[i] grows to new_lens[i] tokens (>= its length):
 * pages are taken for it, the free ones of lowest index in the order of the
 * requests, and entered in its table; lens is set.  ids are distinct.  n up to
 * 65536. */
int moe_kv4_reserve(const moe_kv4_shape *shape, const moe_kv4_seqs *seqs, const int32_t *ids,
                    const int32_t *new_lens, int n, void *scratch, size_t scratch_bytes,
                    uint32_t *err, moe_stream_t stream);

/* moe_kv4_fork: sequence children[i] (which holds nothing) becomes a copy of
 * parents[i].  Full pages are shared (refs + 1); the tokens of a page that the
 * parent has only begun are copied, in every layer, to the lowest free page (its
 * other slots keep what they held).  children are distinct and none is a parent. */
int moe_kv4_fork(void *pages, const moe_kv4_shape *shape, const moe_kv4_seqs *seqs,
                 const int32_t *parents, const int32_t *children, int n, void *scratch,
                 size_t scratch_bytes, uint32_t *err, moe_stream_t stream);

/* moe_kv4_free: the sequences ids[i] (distinct) give their pages back (refs - 1;
 * a page is free at 0), their tables are set to -1 and their lengths to 0. */
int moe_kv4_free(const moe_kv4_shape *shape, const moe_kv4_seqs *seqs, const int32_t *ids, int n,
                 uint32_t *err, moe_stream_t stream);

/* moe_kv4_compact: the U pages in use move to indices 0..U-1: the k-th used page
 * at or above U goes, in every layer, to the k-th free page below U.  refs_out
 * [n_pages] and tables_out ([seqs][table_stride], as tables) receive the new state
 * and may be seqs->refs and seqs->tables themselves; n_used (int32[1]) receives U.
 * Pages that moved keep their old contents as well. */
int moe_kv4_compact(void *pages, const moe_kv4_shape *shape, const moe_kv4_seqs *seqs,
                    int32_t *tables_out, int32_t *refs_out, int32_t *n_used, void *scratch,
                    size_t scratch_bytes, uint32_t *err, moe_stream_t stream);

/* moe_kv4_copy_pages: page dst[i] becomes a copy of page src[i], in every layer
 * (a pair with a negative id is skipped).  No page is both copied to and another
 * pair's source or target. */
int moe_kv4_copy_pages(void *pages, const moe_kv4_shape *shape, const int32_t *src,
                       const int32_t *dst, int n, uint32_t *err, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_KV4_H */
