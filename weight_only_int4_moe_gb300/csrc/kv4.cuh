// Shared by the kernels of the 4-bit paged key/value cache (kv4_*.cu): the
// pool's geometry, the lookup of a token's request and page, and the code and
// scale arithmetic of include/moe_kv4.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "moe_kv4.h"

namespace moe {

constexpr float kKvScaleMin = 6.103515625e-05f;  // 2^-14
constexpr float kKvScaleMax = 2720.0f;           // largest bf16 whose 24-fold fp16 holds
constexpr float kKvSeventh = 1.0f / 7.0f;
constexpr float kKvMax = 7.0f * kKvScaleMax;     // 19040

// One layer of the pool.
struct KvPool {
    uint8_t *base;       // the layer's first page
    int n_pages, hkv, ps;
    uint32_t block;      // bytes of a block: ps * (D + D / 8)
};

struct KvBatch {
    const int32_t *cu_q, *kv_len, *tables;
    int requests, tokens, stride;
};

MOE_DEV void kv_report(uint32_t *err, uint32_t flag) {
    if (err) {
        atomicOr(err, flag);
        atomicAdd(err + 1, 1u);
    }
}

// The request that token t belongs to: the last b with cu_q[b] <= t.  A decode
// batch has one token a request, so b = t is tried first.
MOE_DEV int kv_request_of(const int32_t *cu_q, int requests, int t) {
    const int guess = min(t, requests - 1);
    if (cu_q[guess] <= t && t < cu_q[guess + 1]) return guess;
    int lo = 0, hi = requests - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu_q[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The page of token j of a sequence, or -1 (and a report) where its table has
// none.
MOE_DEV int kv_page_of(const KvBatch &b, const KvPool &p, int request, int j, uint32_t *err) {
    const int e = j / p.ps;
    int page = -1;
    if (e < b.stride) page = b.tables[(size_t)request * b.stride + e];
    if ((unsigned)page >= (unsigned)p.n_pages) {
        kv_report(err, MOE_KV4_DEVERR_PAGE);
        return -1;
    }
    return page;
}

MOE_DEV uint8_t *kv_block(const KvPool &p, int page, int head) {
    return p.base + ((size_t)page * p.hkv + head) * p.block;
}

// n / group for row numbers below 2^26 and groups of up to 64: one multiply by
// magic = floor(2^32 / group) + 1 (whose error stays below n * group < 2^32).
struct GroupDiv {
    uint32_t magic;  // 0: group 1
    int group;
};
MOE_DEV int div_group(int n, GroupDiv g) { return g.magic ? (int)__umulhi((uint32_t)n, g.magic) : n; }

MOE_DEV float kv_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One row's four dimensions added up over several parts, in their order: each
// holds sums o relative to a maximum m and their weight l.  U parts are loaded at
// once (a part at a time would cost a memory round trip each).  at(i): the part's
// row, D sums, then m and l; sl2 > 0 turns scores into powers of two.
template <int D, int U, typename At>
MOE_DEV void add_parts(int n, int d4, float sl2, At at, float &m, float &l, float4 &s) {
    m = -INFINITY;
    l = 0.0f;
    s = make_float4(0, 0, 0, 0);
    for (int i0 = 0; i0 < n; i0 += U) {
        float pm[U], pl[U];
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float *r = at(min(i0 + u, n - 1));
            const float2 ml = *reinterpret_cast<const float2 *>(r + D);
            v[u] = *reinterpret_cast<const float4 *>(r + 4 * d4);
            pm[u] = i0 + u < n ? ml.x : -INFINITY;
            pl[u] = ml.y;
        }
        float nm = m;
#pragma unroll
        for (int u = 0; u < U; ++u) nm = fmaxf(nm, pm[u]);
        const float x = m > -INFINITY ? kv_ex2((m - nm) * sl2) : 0.0f;
        m = nm;
        l *= x;
        s.x *= x, s.y *= x, s.z *= x, s.w *= x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float y = pm[u] > -INFINITY ? kv_ex2((pm[u] - nm) * sl2) : 0.0f;
            l = fmaf(pl[u], y, l);
            s.x = fmaf(v[u].x, y, s.x);
            s.y = fmaf(v[u].y, y, s.y);
            s.z = fmaf(v[u].z, y, s.z);
            s.w = fmaf(v[u].w, y, s.w);
        }
    }
}

// The scale of a group: bf16(amax / 7) in [2^-14, 2720] (also for amax = 0).
MOE_DEV float kv_scale(float amax) {
    const float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(amax, kKvSeventh)));
    return fminf(fmaxf(s, kKvScaleMin), kKvScaleMax);
}

// rint(x / s) limited to -8..7, plus 8; the quotient is the IEEE one.
MOE_DEV uint32_t kv_code(float x, float s) {
    const float r = rintf(__fdiv_rn(x, s));
    return (uint32_t)(int)(fminf(fmaxf(r, -8.0f), 7.0f) + 8.0f);
}

}  // namespace moe
