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

// The index in its sequence of token t, which kv_request_of found in request b.  Negative:
// it has no place there, being before the sequence's first token or, with owned false, a
// row outside every request's range.
MOE_DEV int kv_index_of(const KvBatch &b, int request, int t, bool &owned) {
    const int q1 = b.cu_q[request + 1];
    owned = t >= b.cu_q[request] && t < q1;
    return owned ? b.kv_len[request] - (q1 - t) : -1;
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

// Adds up several parts of the same rows, in their order: each part holds, for a
// row, D sums relative to a maximum, then the maximum m and the weight l.  A whole
// warp takes R rows at a time (D = 64: twice R, half a warp each), a lane four
// dimensions, and requests U parts of all its rows at once: a row or a part at a
// time would cost a memory round trip each.  at(i) is part i (rows of D + 4 floats);
// sl2 > 0 turns scores into powers of two; done(row, d4, m, l, sums) takes a result.
template <int D, int R, int U, typename At, typename Done>
MOE_DEV void add_parts(int n, int row0, float sl2, At at, Done done) {
    constexpr int kLanes = D / 4, kStep = 32 / kLanes;
    const int lane = threadIdx.x & 31, d4 = lane % kLanes, first = row0 + lane / kLanes;
    float m[R], l[R];
    float4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.0f;
        s[r] = make_float4(0, 0, 0, 0);
    }
    for (int i0 = 0; i0 < n; i0 += U) {
        float2 ml[U][R];
        float4 v[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float *p = at(min(i0 + u, n - 1)) + first * (D + 4);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                ml[u][r] = *reinterpret_cast<const float2 *>(p + r * kStep * (D + 4) + D);
                v[u][r] = *reinterpret_cast<const float4 *>(p + r * kStep * (D + 4) + 4 * d4);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float nm = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) nm = fmaxf(nm, ml[u][r].x);  // a part twice: no harm
            const float base = nm > -INFINITY ? nm : 0.0f;
            const float x = kv_ex2((m[r] - base) * sl2);
            m[r] = nm;
            l[r] *= x;
            s[r].x *= x, s[r].y *= x, s[r].z *= x, s[r].w *= x;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float y = i0 + u < n ? kv_ex2((ml[u][r].x - base) * sl2) : 0.0f;
                l[r] = fmaf(ml[u][r].y, y, l[r]);
                s[r].x = fmaf(v[u][r].x, y, s[r].x);
                s[r].y = fmaf(v[u][r].y, y, s[r].y);
                s[r].z = fmaf(v[u][r].z, y, s[r].z);
                s[r].w = fmaf(v[u][r].w, y, s[r].w);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) done(first + r * kStep, d4, m[r], l[r], s[r]);
}

// The scale of a group: bf16(amax / 7) in [2^-14, 2720] (also for amax = 0).
MOE_DEV float kv_scale(float amax) {
    const float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(amax, kKvSeventh)));
    return fminf(fmaxf(s, kKvScaleMin), kKvScaleMax);
}

}  // namespace moe
