// Arguments and launchers of the cache kernels, between kv4_abi.cu and the
// kernels' files.
#pragma once

#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {

struct KvAppendArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const uint16_t *q_weight, *k_weight;
    const float *cos, *sin;
    const int32_t *positions;
    float eps;
    int max_pos, interleaved, q_heads;
    int split;  // warps of a token
    uint16_t *q_out;
    KvPool pool;
    KvBatch batch;
    uint32_t *err;
};

struct KvReadArgs {
    KvPool pool;
    KvBatch batch;
    uint16_t *k_out, *v_out;
    uint32_t *err;
};

// Constants of the unpacking, as kernel parameters: they stay constant-bank operands
// where the compiler would put immediates into registers again for every use, and
// shifts to the left become multiplies of the FMA pipe, which has room where the ALU
// pipe has none.
struct alignas(16) KvConsts {
    uint32_t c4 = 4, c16 = 16, c64 = 64;
    uint32_t nib4 = 0x00F000F0u, magic64 = 0x54005400u;   // a nibble at bits 4..7: fp16 64 + q
    uint32_t nib6 = 0x03C003C0u, magic16 = 0x4C004C00u;   // at bits 6..9: 16 + q
    uint32_t cm24 = 0xCE00CE00u;                          // fp16 pair (-24, -24)
};

// The longest sequence that attention works on, in tokens: what it adds to and takes from
// a token's index (tiles, windows, new tokens) then stays inside an int.
constexpr int kKvMaxLen = INT32_MAX - (1 << 22);

struct KvAttnArgs {
    const uint16_t *q;
    int64_t q_stride;
    KvPool pool;
    KvBatch batch;
    const uint64_t *tree;
    uint16_t *out;
    float *lse;
    float scale_log2;  // scale * log2(e)
    int q_heads, group, window;
    GroupDiv gdiv;
    int rows_lo, rows_hi;  // requests of this many rows (new tokens x group) are the kernel's
    int max_kv, min_units;
    KvConsts k;
    int32_t *counters;     // [CTAs], zero between calls
    float *warp_slots, *cta_slots;
    uint32_t *err;
    bool beside;           // both kernels take part: the decode kernel runs beside the other
    // scale_log2's magnitude (no less than 1e-30), and in units of q . k:
    //  raise: probabilities are relative to a number that lies 2^7 below the row's maximum
    //    (where that was found; it may grow by up to `lag`, 2^8, before they are related to a
    //    new one), so that they fill fp16 up to 2^15.  Relative to the maximum itself, what
    //    lies 2^14 below would lose bits and what lies 2^25 below would be lost, while the
    //    sum counts it: in a long context with one strong token percents of the output.
    //  far: from this magnitude on fp32 holds a score's power of two in steps of an eighth
    //    or more; such rows are related to the maximum itself.
    //  reach: raise + lag.
    float sl2, lag, far, raise, reach;
    // Debug-bounds builds: CTA 0 leaves a tile's copy out (decode kernel, its first warp), or
    // does not say that V's is unpacked (prefill kernel), so that a wait runs out.  -1: none.
    int skip_tile;
};

constexpr int kKvMaxCtas = 160;     // slots of the workspace (a GB300 has 152 SMs)
// Rows of a request (new tokens x group) up to which the decode kernel takes it, which
// works on 16 of them at a time.  Measured, decode against prefill kernel: 10 streams of
// 4000 tokens, 8 kv heads of 128 dimensions, 16, 32, 64 and 128 rows: 29, 41, 66 and
// 118 us against 50, 51, 53 and 57; 32 such streams, 32, 64 and 128 rows: 99, 182 and
// 344 us against 131, 136 and 142; 24 of 2000 tokens, 16 heads of 64, the same rows: 54,
// 98 and 187 us against 68, 70 and 73.
constexpr int kKvFewRows = 48;
constexpr int kKvCounterByte = 256; // the counters' place in the workspace header

// The pool for page management (all layers).
struct KvPages {
    uint8_t *pages;
    int layers, n_pages, hkv, D, ps;
    uint32_t block;
};

cudaError_t launch_kv4_append(KvAppendArgs a, int D, int sms, cudaStream_t s);
cudaError_t launch_kv4_read(const KvReadArgs &a, int D, cudaStream_t s);
// Attention of the requests with few rows; max_rows bounds a request's rows.
size_t kv4_decode_slot_bytes(int D, int ctas);
cudaError_t launch_kv4_decode(KvAttnArgs a, int D, int max_rows, void *slots, int ctas,
                              cudaStream_t s);
// Attention of the requests with many rows (a.rows_lo and up).
size_t kv4_prefill_slot_bytes(int D, int ctas);
cudaError_t launch_kv4_prefill(KvAttnArgs a, int D, void *slots, int ctas, cudaStream_t s);
// fork: a are parents, b children (one page for each parent with a begun page); else
// reserve: a are sequences, b their new lengths.
cudaError_t launch_kv4_take(const KvPages &p, const moe_kv4_seqs &q, const int32_t *a,
                            const int32_t *b, bool fork, int n, void *scratch, uint32_t *err,
                            cudaStream_t s);
cudaError_t launch_kv4_free(const KvPages &p, const moe_kv4_seqs &q, const int32_t *ids, int n,
                            uint32_t *err, cudaStream_t s);
cudaError_t launch_kv4_compact(const KvPages &p, const moe_kv4_seqs &q, int32_t *tables_out,
                               int32_t *refs_out, int32_t *n_used, void *scratch, uint32_t *err,
                               int sms, cudaStream_t s);
cudaError_t launch_kv4_copy(const KvPages &p, const int32_t *src, const int32_t *dst, int n,
                            uint32_t *err, int sms, cudaStream_t s);

}  // namespace moe
