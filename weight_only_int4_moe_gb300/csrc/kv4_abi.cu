// Host side of include/moe_kv4.h: argument checks and launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>
#include <cstdlib>

#include "device.cuh"
#include "kv4_launch.cuh"

using namespace moe;

namespace moe {

// SM count of the current device, MOE_ERR_UNSUPPORTED unless it is sm_103.
int device_sms(int *sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev >= 0 && dev < 64) {
        *sms = known[dev].load(std::memory_order_relaxed);
        if (*sms > 0) return MOE_OK;
    }
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
    if (dev >= 0 && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
    return MOE_OK;
}

}  // namespace moe

namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

bool shape_ok(const moe_kv4_shape *s) {
    return s->layers >= 1 && s->layers <= 1024 && s->n_pages >= 1 && s->n_pages <= (1 << 20) &&
           s->kv_heads >= 1 && s->kv_heads <= 256 && (s->head_dim == 64 || s->head_dim == 128) &&
           (s->page_size == 16 || s->page_size == 32 || s->page_size == 64);
}

bool batch_ok(const moe_kv4_batch *b) {
    return b->requests >= 0 && b->requests <= 65536 && b->tokens >= 0 && b->tokens <= (1 << 20) &&
           b->max_q >= 0 && b->max_kv >= 0 && b->table_stride >= 0 &&
           (b->tokens == 0 || b->requests > 0);
}

uint32_t block_bytes(const moe_kv4_shape *s) {
    return (uint32_t)s->page_size * (uint32_t)(s->head_dim + s->head_dim / 8);
}

// The pieces that every call over a batch checks; MOE_OK with *empty when there
// is nothing to do.
int check_batch(const void *pages, int layer, const moe_kv4_shape *shape,
                const moe_kv4_batch *batch, bool *empty) {
    if (!shape || !batch) return MOE_ERR_NULL;
    if (!shape_ok(shape) || !batch_ok(batch)) return MOE_ERR_SHAPE;
    if (layer < 0 || layer >= shape->layers) return MOE_ERR_SHAPE;
    *empty = batch->tokens == 0;
    if (*empty) return MOE_OK;
    if (!pages || !batch->cu_q || !batch->kv_len || !batch->tables) return MOE_ERR_NULL;
    if (!aligned16(pages)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

KvPool pool_of(const void *pages, int layer, const moe_kv4_shape *s) {
    KvPool p;
    p.block = block_bytes(s);
    p.base = reinterpret_cast<uint8_t *>(const_cast<void *>(pages)) +
             (size_t)layer * s->n_pages * s->kv_heads * p.block;
    p.n_pages = s->n_pages;
    p.hkv = s->kv_heads;
    p.ps = s->page_size;
    return p;
}

KvBatch batch_of(const moe_kv4_batch *b) {
    return KvBatch{b->cu_q, b->kv_len, b->tables, b->requests, b->tokens, b->table_stride};
}

KvPages pages_of(void *pages, const moe_kv4_shape *s) {
    return KvPages{reinterpret_cast<uint8_t *>(pages), s->layers,    s->n_pages, s->kv_heads,
                   s->head_dim,                        s->page_size, block_bytes(s)};
}

int check_seqs(const moe_kv4_shape *shape, const moe_kv4_seqs *q, int n, bool lens) {
    if (!shape || !q) return MOE_ERR_NULL;
    if (!shape_ok(shape)) return MOE_ERR_SHAPE;
    if (q->seqs < 1 || q->seqs > 65536 || q->table_stride < 1) return MOE_ERR_SHAPE;
    if (n < 0 || n > 65536) return MOE_ERR_SHAPE;
    if (!q->tables || !q->refs || (lens && !q->lens)) return MOE_ERR_NULL;
    return MOE_OK;
}

inline int done(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline cudaStream_t str(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

size_t moe_kv4_block_bytes(const moe_kv4_shape *shape) {
    return shape && shape_ok(shape) ? block_bytes(shape) : 0;
}

size_t moe_kv4_pool_bytes(const moe_kv4_shape *shape) {
    return moe_kv4_block_bytes(shape) *
           (shape && shape_ok(shape) ? (size_t)shape->layers * shape->n_pages * shape->kv_heads : 0);
}

int moe_kv4_append(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                   const uint16_t *v, int64_t v_stride, const uint16_t *q_weight,
                   const uint16_t *k_weight, float eps, const float *cos, const float *sin,
                   const int32_t *positions, int max_pos, int interleaved, int q_heads,
                   uint16_t *q_out, void *pages, int layer, const moe_kv4_shape *shape,
                   const moe_kv4_batch *batch, uint32_t *err, moe_stream_t stream) {
    bool empty;
    int rc = check_batch(pages, layer, shape, batch, &empty);
    if (rc != MOE_OK) return rc;
    const int D = shape->head_dim;
    if (!q) q_heads = 0;
    if (q_heads < 0 || q_heads > 1024 || (q && q_heads == 0)) return MOE_ERR_SHAPE;
    if ((!cos) != (!sin)) return MOE_ERR_NULL;
    if (cos && max_pos < 1) return MOE_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return MOE_ERR_SHAPE;
    if (interleaved != 0 && interleaved != 1) return MOE_ERR_SHAPE;
    if (empty) return MOE_OK;
    if (!k || !v || (q && !q_out)) return MOE_ERR_NULL;
    if ((q && (q_stride < (int64_t)q_heads * D || q_stride % 8)) ||
        k_stride < (int64_t)shape->kv_heads * D || k_stride % 8 ||
        v_stride < (int64_t)shape->kv_heads * D || v_stride % 8)
        return MOE_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_weight) ||
        !aligned16(k_weight) || !aligned16(cos) || !aligned16(sin) || !aligned16(q_out))
        return MOE_ERR_ALIGN;
    int sms;
    rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    KvAppendArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    a.eps = eps;
    a.max_pos = max_pos;
    a.interleaved = interleaved;
    a.q_heads = q_heads;
    a.q_out = q_out;
    a.pool = pool_of(pages, layer, shape);
    a.batch = batch_of(batch);
    a.err = err;
    return done(launch_kv4_append(a, D, sms, str(stream)));
}

int moe_kv4_read(const void *pages, int layer, const moe_kv4_shape *shape,
                 const moe_kv4_batch *batch, uint16_t *k_out, uint16_t *v_out, uint32_t *err,
                 moe_stream_t stream) {
    bool empty;
    int rc = check_batch(pages, layer, shape, batch, &empty);
    if (rc != MOE_OK) return rc;
    if (empty) return MOE_OK;
    if (!k_out && !v_out) return MOE_OK;
    if (!aligned16(k_out) || !aligned16(v_out)) return MOE_ERR_ALIGN;
    int sms;
    rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    KvReadArgs a{};
    a.pool = pool_of(pages, layer, shape);
    a.batch = batch_of(batch);
    a.k_out = k_out;
    a.v_out = v_out;
    a.err = err;
    return done(launch_kv4_read(a, shape->head_dim, str(stream)));
}

size_t moe_kv4_workspace_bytes(const moe_kv4_shape *shape, int q_heads) {
    if (!shape || !shape_ok(shape) || q_heads < 1 || q_heads % shape->kv_heads ||
        q_heads / shape->kv_heads > 64)
        return 0;
    const size_t few = kv4_decode_slot_bytes(shape->head_dim, kKvMaxCtas);
    const size_t many = kv4_prefill_slot_bytes(shape->head_dim, kKvMaxCtas);
    return MOE_KV4_WS_HEADER + few + many;
}

int moe_kv4_attention(const uint16_t *q, int64_t q_stride, int q_heads, const void *pages,
                      int layer, const moe_kv4_shape *shape, const moe_kv4_batch *batch,
                      float scale, int window, const uint64_t *tree, uint16_t *out, float *lse,
                      void *workspace, size_t workspace_bytes, moe_stream_t stream) {
    bool empty;
    int rc = check_batch(pages, layer, shape, batch, &empty);
    if (rc != MOE_OK) return rc;
    if (!moe_kv4_workspace_bytes(shape, q_heads)) return MOE_ERR_SHAPE;
    const float scale_log2 = scale * 1.4426950408889634f;
    if (window < 0 || !std::isfinite(scale_log2)) return MOE_ERR_SHAPE;
    if (tree && batch->max_q > 64) return MOE_ERR_SHAPE;
    if (empty) return MOE_OK;
    if (!q || !out || !workspace) return MOE_ERR_NULL;
    if (q_stride < (int64_t)q_heads * shape->head_dim || q_stride % 8) return MOE_ERR_SHAPE;
    if (workspace_bytes < moe_kv4_workspace_bytes(shape, q_heads)) return MOE_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || ((uintptr_t)lse & 3u) ||
        ((uintptr_t)tree & 7u))
        return MOE_ERR_ALIGN;
    int sms;
    rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    KvAttnArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.pool = pool_of(pages, layer, shape);
    a.batch = batch_of(batch);
    a.tree = tree;
    a.out = out;
    a.lse = lse;
    a.scale_log2 = scale_log2;
    a.sl2 = std::fmax(std::fabs(a.scale_log2), 1e-30f);
    a.lag = 8.0f / a.sl2;
    a.far = 1048576.0f / a.sl2;
    a.raise = 7.0f / a.sl2;
    a.reach = 15.0f / a.sl2;
    a.q_heads = q_heads;
    a.group = q_heads / shape->kv_heads;
    a.gdiv.group = a.group;
    a.gdiv.magic = a.group == 1 ? 0u : (uint32_t)((1ull << 32) / a.group + 1);
    a.window = window > kKvMaxLen ? 0 : window;  // no sequence is longer
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    a.err = reinterpret_cast<uint32_t *>(ws);
    a.max_kv = batch->max_kv;
    a.skip_tile = -1;
#ifdef MOE_DEBUG_BOUNDS
    if (const char *v = getenv("MOE_KV4_DEBUG_SKIP_TILE")) a.skip_tile = atoi(v);
#endif
    // Requests of up to kKvFewRows rows go to the decode kernel, others to the
    // prefill kernel; where all have the same number of new tokens one is enough.
    const int ctas = sms < kKvMaxCtas ? sms : kKvMaxCtas;
    uint8_t *slots = ws + MOE_KV4_WS_HEADER;
    const long long most = (long long)batch->max_q * a.group;
    const bool even = (long long)batch->requests * batch->max_q == batch->tokens;
    const bool few = most <= kKvFewRows || !even, many = most > kKvFewRows;
    // the kernels count their units of work in 32 bits
    const double few_rows = most < kKvFewRows ? (double)most : (double)kKvFewRows;
    const double tiles = batch->max_kv / 64.0 + 8.0;
    if ((few && batch->requests * (few_rows / 8 + 1) * shape->kv_heads * tiles > 4e9) ||
        (many && ((double)batch->tokens * a.group / 256 + batch->requests) * shape->kv_heads * tiles > 4e9))
        return MOE_ERR_SHAPE;
    cudaStream_t s = str(stream);
    // Both: the prefill kernel first; the decode kernel's blocks then start on the SMs
    // that it leaves, with slots and counters of their own.
    a.beside = few && many;
    if (many) {
        a.counters = reinterpret_cast<int32_t *>(ws + kKvCounterByte) + kKvMaxCtas;
        a.rows_lo = few ? kKvFewRows + 1 : 1;
        a.rows_hi = INT32_MAX;
        const cudaError_t e = launch_kv4_prefill(
            a, shape->head_dim, slots + kv4_decode_slot_bytes(shape->head_dim, kKvMaxCtas), ctas, s);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (few) {
        a.counters = reinterpret_cast<int32_t *>(ws + kKvCounterByte);
        a.rows_lo = 1;
        a.rows_hi = many ? kKvFewRows : INT32_MAX;
        const cudaError_t e = launch_kv4_decode(
            a, shape->head_dim, most < kKvFewRows ? (int)most : kKvFewRows, slots, ctas, s);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

size_t moe_kv4_scratch_bytes(const moe_kv4_shape *shape, int n) {
    if (!shape || !shape_ok(shape) || n < 0 || n > 65536) return 0;
    return ((size_t)3 * shape->n_pages + 2 * (size_t)n + 16) * 4;
}

static int take(void *pages, const moe_kv4_shape *shape, const moe_kv4_seqs *seqs,
                const int32_t *a, const int32_t *b, bool fork, int n, void *scratch,
                size_t scratch_bytes, uint32_t *err, moe_stream_t stream) {
    int rc = check_seqs(shape, seqs, n, true);
    if (rc != MOE_OK) return rc;
    if (n == 0) return MOE_OK;
    if (!a || !b || !scratch || (fork && !pages)) return MOE_ERR_NULL;
    if (scratch_bytes < moe_kv4_scratch_bytes(shape, n)) return MOE_ERR_WORKSPACE;
    if (!aligned16(pages) || !aligned16(scratch)) return MOE_ERR_ALIGN;
    int sms;
    rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    return done(
        launch_kv4_take(pages_of(pages, shape), *seqs, a, b, fork, n, scratch, err, str(stream)));
}

int moe_kv4_reserve(const moe_kv4_shape *shape, const moe_kv4_seqs *seqs, const int32_t *ids,
                    const int32_t *new_lens, int n, void *scratch, size_t scratch_bytes,
                    uint32_t *err, moe_stream_t stream) {
    return take(nullptr, shape, seqs, ids, new_lens, false, n, scratch, scratch_bytes, err, stream);
}

int moe_kv4_fork(void *pages, const moe_kv4_shape *shape, const moe_kv4_seqs *seqs,
                 const int32_t *parents, const int32_t *children, int n, void *scratch,
                 size_t scratch_bytes, uint32_t *err, moe_stream_t stream) {
    return take(pages, shape, seqs, parents, children, true, n, scratch, scratch_bytes, err, stream);
}

int moe_kv4_free(const moe_kv4_shape *shape, const moe_kv4_seqs *seqs, const int32_t *ids, int n,
                 uint32_t *err, moe_stream_t stream) {
    int rc = check_seqs(shape, seqs, n, true);
    if (rc != MOE_OK) return rc;
    if (n == 0) return MOE_OK;
    if (!ids) return MOE_ERR_NULL;
    int sms;
    rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    return done(launch_kv4_free(pages_of(nullptr, shape), *seqs, ids, n, err, str(stream)));
}

int moe_kv4_compact(void *pages, const moe_kv4_shape *shape, const moe_kv4_seqs *seqs,
                    int32_t *tables_out, int32_t *refs_out, int32_t *n_used, void *scratch,
                    size_t scratch_bytes, uint32_t *err, moe_stream_t stream) {
    int rc = check_seqs(shape, seqs, 0, false);
    if (rc != MOE_OK) return rc;
    if (!pages || !tables_out || !refs_out || !n_used || !scratch) return MOE_ERR_NULL;
    if (scratch_bytes < moe_kv4_scratch_bytes(shape, 0)) return MOE_ERR_WORKSPACE;
    if (!aligned16(pages) || !aligned16(scratch)) return MOE_ERR_ALIGN;
    int sms;
    rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    return done(launch_kv4_compact(pages_of(pages, shape), *seqs, tables_out, refs_out, n_used,
                                   scratch, err, sms, str(stream)));
}

int moe_kv4_copy_pages(void *pages, const moe_kv4_shape *shape, const int32_t *src,
                       const int32_t *dst, int n, uint32_t *err, moe_stream_t stream) {
    if (!shape) return MOE_ERR_NULL;
    if (!shape_ok(shape) || n < 0 || n > shape->n_pages) return MOE_ERR_SHAPE;
    if (n == 0) return MOE_OK;
    if (!pages || !src || !dst) return MOE_ERR_NULL;
    if (!aligned16(pages)) return MOE_ERR_ALIGN;
    int sms;
    const int rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    return done(launch_kv4_copy(pages_of(pages, shape), src, dst, n, err, sms, str(stream)));
}

}  // extern "C"
