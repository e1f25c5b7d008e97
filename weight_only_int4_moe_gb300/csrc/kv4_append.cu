// Appending to and reading from the 4-bit cache (include/moe_kv4.h).
//
// append: per head row of D values, fp32 throughout,
//   y = x * (1 / sqrt(sum x^2 / D + eps)) * w,  then the rotation of its D/2 pairs,
// the q rows rounded to bf16, the k and v rows quantised into their page.  Bound
// by memory: it reads T (Hq + 2 Hkv) D bf16 values and writes T Hq D of them plus
// 9/16 byte per cached value.  A row belongs to D/16 lanes, each holding eight
// values from either half of the row: both members of every rotation pair
// (i, i + D/2) and (2i, 2i + 1) are in one lane, loads are 16 bytes, and a lane's
// eight values are exactly one 32-bit word of the K row, so the codes need no
// exchange.  Only the sum of squares (a butterfly over the row's lanes, whose
// order does not depend on the lane) and the group maximum (four lanes) do.
#include "kv4.cuh"
#include "kv4_launch.cuh"

namespace moe {

namespace {

MOE_DEV void unpack8(const uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

MOE_DEV uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

MOE_DEV void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// (a, b) -> (a c - b s, b c + a s), every operation rounded on its own.
MOE_DEV void turn(float &a, float &b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// A row's eight values of one group of 32 (four lanes hold a group): codes and
// scale, saturating what the format cannot hold.
MOE_DEV float quantise8(float (&x)[8], uint32_t (&q)[8], bool &bad) {
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (!(fabsf(x[j]) <= kKvMax)) {
            bad = true;
            x[j] = x[j] != x[j] ? 0.0f : copysignf(kKvMax, x[j]);
        }
        amax = fmaxf(amax, fabsf(x[j]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float s = kv_scale(amax);
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = kv_code(x[j], s);
    return s;
}

template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const KvAppendArgs a) {
    constexpr int kLanes = D / 16;      // lanes of a row
    constexpr int kRows = 32 / kLanes;  // rows of a warp
    constexpr int NG = D / 32;
    pdl_wait();
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const int heads = a.q_heads + 2 * a.pool.hkv;
    const int rows = a.batch.tokens * heads;
    const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    int row = warp * kRows + lane / kLanes;
    if (warp * kRows >= rows) return;
    const bool live = row < rows;  // lanes past the end repeat the last row and write nothing
    row = min(row, rows - 1);
    const int t = row / heads, h = row - t * heads;
    const int kind = h < a.q_heads ? 0 : h < a.q_heads + a.pool.hkv ? 1 : 2;  // q, k, v
    const int hk = kind == 0 ? h : kind == 1 ? h - a.q_heads : h - a.q_heads - a.pool.hkv;
    const uint16_t *src = kind == 0   ? a.q + (size_t)t * a.q_stride
                          : kind == 1 ? a.k + (size_t)t * a.k_stride
                                      : a.v + (size_t)t * a.v_stride;
    src += (size_t)hk * D + 8 * l;
    float x[8], y[8];
    unpack8(*reinterpret_cast<const uint4 *>(src), x);
    unpack8(*reinterpret_cast<const uint4 *>(src + D / 2), y);

    // the token's place: its request and index there
    const bool place = kind != 0 || (a.cos && !a.positions);
    int b = 0, at = 0;
    if (place) {
        b = kv_request_of(a.batch.cu_q, a.batch.requests, t);
        at = a.batch.kv_len[b] - (a.batch.cu_q[b + 1] - t);
    }

    // sum of squares of the row, in the documented order
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = __fadd_rn(__fmul_rn(x[j], x[j]), __fmul_rn(y[j], y[j]));
    float sum = __fadd_rn(__fadd_rn(__fadd_rn(s[0], s[4]), __fadd_rn(s[2], s[6])),
                          __fadd_rn(__fadd_rn(s[1], s[5]), __fadd_rn(s[3], s[7])));
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, m));

    const uint16_t *w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    if (w) {
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / D), a.eps)));
        float g[8];
        unpack8(*reinterpret_cast<const uint4 *>(w + 8 * l), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], r), g[j]);
        unpack8(*reinterpret_cast<const uint4 *>(w + D / 2 + 8 * l), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(__fmul_rn(y[j], r), g[j]);
    }
    if (kind < 2 && a.cos) {
        int pos = a.positions ? a.positions[t] : at;
        if (pos < 0 || pos >= a.max_pos) {
            if (l == 0 && live) kv_report(a.err, MOE_KV4_DEVERR_POSITION);
            pos = min(max(pos, 0), a.max_pos - 1);
        }
        const float *cs = a.cos + (size_t)pos * (D / 2), *sn = a.sin + (size_t)pos * (D / 2);
        float c[8], z[8];
        if (!a.interleaved) {
            load8(cs + 8 * l, c);
            load8(sn + 8 * l, z);
#pragma unroll
            for (int j = 0; j < 8; ++j) turn(x[j], y[j], c[j], z[j]);
        } else {
            *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(cs + 4 * l);
            *reinterpret_cast<float4 *>(c + 4) =
                *reinterpret_cast<const float4 *>(cs + D / 4 + 4 * l);
            *reinterpret_cast<float4 *>(z) = *reinterpret_cast<const float4 *>(sn + 4 * l);
            *reinterpret_cast<float4 *>(z + 4) =
                *reinterpret_cast<const float4 *>(sn + D / 4 + 4 * l);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                turn(x[2 * j], x[2 * j + 1], c[j], z[j]);
                turn(y[2 * j], y[2 * j + 1], c[4 + j], z[4 + j]);
            }
        }
    }

    if (kind == 0 && live) {
        uint16_t *dst = a.q_out + ((size_t)t * a.q_heads + hk) * D + 8 * l;
        *reinterpret_cast<uint4 *>(dst) = pack8(x);
        *reinterpret_cast<uint4 *>(dst + D / 2) = pack8(y);
    }
    // a warp with no row of k or v is done; in a mixed one the rows of q take
    // part in the shuffles below
    if (!__any_sync(0xffffffffu, kind != 0)) return;
    uint32_t qx[8], qy[8];
    bool bad = false;
    const float sx = quantise8(x, qx, bad), sy = quantise8(y, qy, bad);
    if (kind == 0 || !live) return;
    if (at < 0) return;  // more new tokens than the sequence's length
    const int page = kv_page_of(a.batch, a.pool, b, at, l == 0 ? a.err : nullptr);
    if (page < 0) return;
    if (bad) kv_report(a.err, MOE_KV4_DEVERR_RANGE);
    const int ps = a.pool.ps, slot = at % ps;
    uint8_t *blk = kv_block(a.pool, page, hk);
    uint8_t *codes = blk + (kind == 1 ? 0 : ps * (D / 2)) + slot * (D / 2);
    uint16_t *sc = reinterpret_cast<uint16_t *>(blk + ps * D) + (kind == 1 ? 0 : ps * NG) + slot * NG;
    const int tq = l & 3, G = l >> 2, G2 = NG / 2 + G;  // the lane's eighth of its two groups
    if (kind == 1) {
        uint32_t wx = 0, wy = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wx |= qx[2 * i] << (4 * i) | qx[2 * i + 1] << (16 + 4 * i);
            wy |= qy[2 * i] << (4 * i) | qy[2 * i + 1] << (16 + 4 * i);
        }
        reinterpret_cast<uint32_t *>(codes)[tq * NG + G] = wx;
        reinterpret_cast<uint32_t *>(codes)[tq * NG + G2] = wy;
    } else {
        uint16_t *piece = reinterpret_cast<uint16_t *>(codes);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t px = 0, py = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                px |= qx[4 * u + i] << (4 * i);
                py |= qy[4 * u + i] << (4 * i);
            }
            piece[(2 * tq + u) * NG + G] = (uint16_t)px;
            piece[(2 * tq + u) * NG + G2] = (uint16_t)py;
        }
    }
    if (tq == 0) {
        sc[G] = __half_as_ushort(__float2half_rn(sx));
        sc[G2] = __half_as_ushort(__float2half_rn(sy));
    }
}

// One row (token, head, K or V) per D/16 lanes, as in the append.
template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const KvReadArgs a) {
    constexpr int kLanes = D / 16, NG = D / 32;
    pdl_wait();
    const int hkv = a.pool.hkv, ps = a.pool.ps;
    const int row = (blockIdx.x * blockDim.x + threadIdx.x) / kLanes, l = threadIdx.x % kLanes;
    if (row >= a.batch.tokens * hkv) return;
    const bool key = blockIdx.y == 0;
    uint16_t *dst = key ? a.k_out : a.v_out;
    if (!dst) return;
    const int t = row / hkv, h = row - t * hkv;
    const int b = kv_request_of(a.batch.cu_q, a.batch.requests, t);
    const int at = a.batch.kv_len[b] - (a.batch.cu_q[b + 1] - t);
    const int page = at < 0 ? -1 : kv_page_of(a.batch, a.pool, b, at, l == 0 ? a.err : nullptr);
    dst += (size_t)row * D + 8 * l;
    if (page < 0) {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(dst + D / 2) = make_uint4(0, 0, 0, 0);
        return;
    }
    const int slot = at % ps, tq = l & 3;
    const uint8_t *blk = kv_block(a.pool, page, h);
    const uint8_t *codes = blk + (key ? 0 : ps * (D / 2)) + slot * (D / 2);
    const __half *sc = reinterpret_cast<const __half *>(blk + ps * D) + (key ? 0 : ps * NG) + slot * NG;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int G = (l >> 2) + u * (NG / 2);
        const __half s = sc[G];
        int q[8];
        if (key) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(codes)[tq * NG + G];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[2 * i] = (w >> (4 * i)) & 15;
                q[2 * i + 1] = (w >> (16 + 4 * i)) & 15;
            }
        } else {
            const uint16_t *piece = reinterpret_cast<const uint16_t *>(codes);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w = piece[(2 * tq + e) * NG + G];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[4 * e + i] = (w >> (4 * i)) & 15;
            }
        }
        __half2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = __hmul2(__halves2half2(__int2half_rn(q[2 * i] - 8), __int2half_rn(q[2 * i + 1] - 8)),
                           __half2half2(s));
        *reinterpret_cast<uint4 *>(dst + u * (D / 2)) = *reinterpret_cast<const uint4 *>(o);
    }
}

}  // namespace

cudaError_t launch_kv4_append(const KvAppendArgs &a, int D, cudaStream_t s) {
    const long long rows = (long long)a.batch.tokens * (a.q_heads + 2 * a.pool.hkv);
    const int per_block = 256 / (D / 16);
    auto c = pdl_config((unsigned)((rows + per_block - 1) / per_block), 256, 0, s);
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return D == 128 ? cudaLaunchKernelEx(&c, kv4_append_kernel<128>, a)
                    : cudaLaunchKernelEx(&c, kv4_append_kernel<64>, a);
}

cudaError_t launch_kv4_read(const KvReadArgs &a, int D, cudaStream_t s) {
    const long long rows = (long long)a.batch.tokens * a.pool.hkv;
    const int per_block = 256 / (D / 16);
    auto c = pdl_config((unsigned)((rows + per_block - 1) / per_block), 256, 0, s);
    c.gridDim.y = 2;
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return D == 128 ? cudaLaunchKernelEx(&c, kv4_read_kernel<128>, a)
                    : cudaLaunchKernelEx(&c, kv4_read_kernel<64>, a);
}

}  // namespace moe
