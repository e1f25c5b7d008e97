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
// order does not depend on the lane) and the group maximum (four lanes) do.  A warp
// stays with one token and walks its heads, so that the token's place, its rotation
// and the weights are read once; where there are few tokens several warps share one.
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
// scale.  limited: some value is beyond the format or not finite; such values are
// saturated (NaN: 0).  The code is rint(x / s) of the IEEE quotient; x * (1/s) is
// within 2^-19 of it (|x / s| <= 8), so only a product that close to the middle
// between two codes needs the division.
MOE_DEV float quantise8(float (&x)[8], uint32_t (&q)[8], bool limited) {
    if (limited) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!(fabsf(x[j]) <= kKvMax)) x[j] = x[j] != x[j] ? 0.0f : copysignf(kKvMax, x[j]);
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float s = kv_scale(amax), inv = __frcp_rn(s);
    bool near = false;
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float p = x[j] * inv;
        r[j] = rintf(p);
        near |= fabsf(p - r[j]) > 0.5f - 0x1p-18f;
    }
    if (near) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = rintf(__fdiv_rn(x[j], s));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (uint32_t)(int)(fminf(fmaxf(r[j], -8.0f), 7.0f) + 8.0f);
    return s;
}

template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const KvAppendArgs a) {
    constexpr int kLanes = D / 16;      // lanes of a row
    constexpr int kRows = 32 / kLanes;  // rows of a warp
    constexpr int NG = D / 32;
    pdl_wait();
    const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
    const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int t = warp / a.split, share = warp - t * a.split;
    if (t >= a.batch.tokens) return;
    const int hkv = a.pool.hkv, ps = a.pool.ps;
    // the token's steps of kRows heads: q, then k, then v; this warp's part of them
    const int nq = (a.q_heads + kRows - 1) / kRows, nk = (hkv + kRows - 1) / kRows;
    const int steps = nq + 2 * nk;
    const int from = steps * share / a.split, to = steps * (share + 1) / a.split;
    auto source = [&](int step, int &kind, int &head) -> const uint16_t * {
        kind = step < nq ? 0 : step < nq + nk ? 1 : 2;  // q, k, v
        head = (step - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * kRows + sub;
        const uint16_t *p = kind == 0   ? a.q + (size_t)t * a.q_stride
                            : kind == 1 ? a.k + (size_t)t * a.k_stride
                                        : a.v + (size_t)t * a.v_stride;
        // lanes past the last head repeat it and write nothing
        return p + (size_t)min(head, (kind == 0 ? a.q_heads : hkv) - 1) * D + 8 * l;
    };
    int kind, head;
    const uint16_t *src = source(from, kind, head);
    uint4 nx = *reinterpret_cast<const uint4 *>(src), ny = *reinterpret_cast<const uint4 *>(src + D / 2);

    // the token's place, its rotation and the weights
    const int b = kv_request_of(a.batch.cu_q, a.batch.requests, t);
    const int at = a.batch.kv_len[b] - (a.batch.cu_q[b + 1] - t);
    int page = -1;
    // more new tokens than the sequence's length: not stored
    if (to > nq && at >= 0) page = kv_page_of(a.batch, a.pool, b, at, lane == 0 && to == steps ? a.err : nullptr);
    const int slot = at >= 0 ? at % ps : 0;
    float c[8], z[8];
    if (a.cos && from < nq + nk) {
        int pos = a.positions ? a.positions[t] : at;
        if (pos < 0 || pos >= a.max_pos) {
            if (lane == 0 && share == 0) kv_report(a.err, MOE_KV4_DEVERR_POSITION);
            pos = min(max(pos, 0), a.max_pos - 1);
        }
        const float *cs = a.cos + (size_t)pos * (D / 2), *sn = a.sin + (size_t)pos * (D / 2);
        if (!a.interleaved) {
            load8(cs + 8 * l, c);
            load8(sn + 8 * l, z);
        } else {
            // pairs of the row's first half, then of its second
            *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(cs + 4 * l);
            *reinterpret_cast<float4 *>(c + 4) = *reinterpret_cast<const float4 *>(cs + D / 4 + 4 * l);
            *reinterpret_cast<float4 *>(z) = *reinterpret_cast<const float4 *>(sn + 4 * l);
            *reinterpret_cast<float4 *>(z + 4) = *reinterpret_cast<const float4 *>(sn + D / 4 + 4 * l);
        }
    }
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    int weights_of = -1;  // the kind whose weights w0, w1 are

    for (int step = from; step < to; ++step) {
        const int kd = kind, hd = head;
        float x[8], y[8];
        unpack8(nx, x);
        unpack8(ny, y);
        if (step + 1 < to) {
            src = source(step + 1, kind, head);
            nx = *reinterpret_cast<const uint4 *>(src);
            ny = *reinterpret_cast<const uint4 *>(src + D / 2);
        }
        const uint16_t *w = kd == 0 ? a.q_weight : kd == 1 ? a.k_weight : nullptr;
        if (w) {
            if (weights_of != kd) {
                weights_of = kd;
                w0 = *reinterpret_cast<const uint4 *>(w + 8 * l);
                w1 = *reinterpret_cast<const uint4 *>(w + D / 2 + 8 * l);
            }
            // sum of squares of the row, in the documented order
            float s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = __fadd_rn(__fmul_rn(x[j], x[j]), __fmul_rn(y[j], y[j]));
            float sum = __fadd_rn(__fadd_rn(__fadd_rn(s[0], s[4]), __fadd_rn(s[2], s[6])),
                                  __fadd_rn(__fadd_rn(s[1], s[5]), __fadd_rn(s[3], s[7])));
#pragma unroll
            for (int m = 1; m < kLanes; m <<= 1)
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, m));
            const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / D), a.eps)));
            float g[8];
            unpack8(w0, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], r), g[j]);
            unpack8(w1, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(__fmul_rn(y[j], r), g[j]);
        }
        if (kd < 2 && a.cos) {
            if (!a.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) turn(x[j], y[j], c[j], z[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    turn(x[2 * j], x[2 * j + 1], c[j], z[j]);
                    turn(y[2 * j], y[2 * j + 1], c[4 + j], z[4 + j]);
                }
            }
        }
        if (kd == 0) {
            if (hd < a.q_heads) {
                uint16_t *dst = a.q_out + ((size_t)t * a.q_heads + hd) * D + 8 * l;
                *reinterpret_cast<uint4 *>(dst) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + D / 2) = pack8(y);
            }
            continue;
        }
        // 0 * v is 0 for finite values and NaN for others
        float odd = 0.0f, big = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            odd = fmaf(0.0f, x[j], fmaf(0.0f, y[j], odd));
            big = fmaxf(big, fmaxf(fabsf(x[j]), fabsf(y[j])));
        }
        const bool limited = odd != 0.0f || big > kKvMax;
        uint32_t qx[8], qy[8];
        const float sx = quantise8(x, qx, limited), sy = quantise8(y, qy, limited);
        const bool mine = hd < hkv && page >= 0;
        if (limited && mine) kv_report(a.err, MOE_KV4_DEVERR_RANGE);
        // the lane's eighth of its two groups G and NG/2 + G
        const int tq = l & 3, G = l >> 2, G2 = NG / 2 + G;
        uint32_t first, second;
        if (kd == 1) {
            // K words (tq, G); D = 128: lanes four apart exchange one, so that each
            // stores two neighbours
            uint32_t wx = 0, wy = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wx |= qx[2 * i] << (4 * i) | qx[2 * i + 1] << (16 + 4 * i);
                wy |= qy[2 * i] << (4 * i) | qy[2 * i + 1] << (16 + 4 * i);
            }
            first = wx, second = wy;
            if (D == 128) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, G ? wx : wy, 4);
                first = G ? got : wx;
                second = G ? wy : got;
            }
        } else {
            // V pieces g = 2 tq, 2 tq + 1 of both groups; D = 128: of lanes four apart
            // one stores g = 2 tq of all four groups, the other g = 2 tq + 1
            uint32_t p[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                p[u] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[u] |= qx[4 * u + i] << (4 * i) | qy[4 * u + i] << (16 + 4 * i);
            }
            first = p[0], second = p[1];
            if (D == 128) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, G ? p[0] : p[1], 4);
                const uint32_t even = G ? got : p[0], odd_g = G ? p[1] : got;  // groups 0, 2 and 1, 3
                first = __byte_perm(even, odd_g, 0x5410);
                second = __byte_perm(even, odd_g, 0x7632);
            }
        }
        if (!mine) continue;
        uint8_t *blk = kv_block(a.pool, page, hd);
        uint8_t *codes = blk + (kd == 1 ? 0 : ps * (D / 2)) + slot * (D / 2);
        uint16_t *sc = reinterpret_cast<uint16_t *>(blk + ps * D) + (kd == 1 ? 0 : ps * NG) + slot * NG;
        // D = 128: K word pairs (tq, 0..1) and (tq, 2..3), V pieces of g = 2 tq + G;
        // D = 64: both of the lane's words
        *reinterpret_cast<uint2 *>(codes + (D == 128 ? 16 * tq + 8 * G : 8 * tq)) =
            make_uint2(first, second);
        if (tq == 0) {
            sc[G] = __half_as_ushort(__float2half_rn(sx));
            sc[G2] = __half_as_ushort(__float2half_rn(sy));
        }
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

cudaError_t launch_kv4_append(KvAppendArgs a, int D, int sms, cudaStream_t s) {
    // as many warps as fill the SMs, where the tokens' steps allow it
    const int rows = 32 / (D / 16);
    const int steps = (a.q_heads + rows - 1) / rows + 2 * ((a.pool.hkv + rows - 1) / rows);
    const long long want = 32ll * sms;
    const long long split = (want + a.batch.tokens - 1) / a.batch.tokens;
    a.split = (int)(split < steps ? split : steps);
    const long long warps = (long long)a.batch.tokens * a.split;
    auto c = pdl_config((unsigned)((warps + 7) / 8), 256, 0, s);
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
