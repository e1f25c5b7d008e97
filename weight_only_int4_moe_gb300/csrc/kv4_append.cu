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
//
// Measured: 6800 tokens of 56 + 8 + 8 heads of 128: 56 us for the 236 MB that append
// itself touches, 4.2 TB/s of the 6.8 that a copy reaches; with the read of what it wrote
// 67 us.  One token of 32 + 8 + 8 heads: 6 us for both, two launches.  The issue slots
// are 61 % busy with the 21 warps that 80 registers a thread allow, the rest waits for
// loads; two heads of a warp are in flight at a time.
#include "kv4.cuh"
#include "kv4_launch.cuh"

namespace moe {

namespace {

// Two floats in one register pair: each is rounded on its own, as by the scalar
// operations, in half the instructions.  A product that is added up next is made by
// prod2: the compiler fuses a packed product with the sum behind it (the scalar
// intrinsics are never fused), and the sum would then see it unrounded.
MOE_DEV uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
MOE_DEV float2 both(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
MOE_DEV uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
MOE_DEV uint64_t prod2(uint64_t a, uint64_t b) {
    const float2 x = both(a), y = both(b);
    return pair(__fmul_rn(x.x, y.x), __fmul_rn(x.y, y.y));
}
MOE_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// a - b: b * -1 is exact, so the one rounding is the difference's.
MOE_DEV uint64_t sub2(uint64_t a, uint64_t b, uint64_t minus1) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(minus1), "l"(a));
    return r;
}
MOE_DEV void unpack8(const uint4 v, uint64_t (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
MOE_DEV uint4 pack8(const uint64_t (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = both(x[i]);
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
MOE_DEV void load8(const float *p, uint64_t (&x)[4]) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// Pairs (a, b) -> (a c - b s, b c + a s), two at a time.
MOE_DEV void turn2(uint64_t &a, uint64_t &b, uint64_t c, uint64_t s, uint64_t minus1) {
    const uint64_t x = sub2(prod2(a, c), prod2(b, s), minus1);
    b = add2(prod2(b, c), prod2(a, s));
    a = x;
}
// One pair whose members are the two halves of v.
MOE_DEV uint64_t turn1(uint64_t v, float c, float s) {
    const float2 f = both(v);
    return pair(__fsub_rn(__fmul_rn(f.x, c), __fmul_rn(f.y, s)),
                __fadd_rn(__fmul_rn(f.y, c), __fmul_rn(f.x, s)));
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

// Where a token's k and v rows go.
struct Place {
    uint8_t *page;  // its page's first block; null: nowhere
    int slot;
};

// The steps [from, to) of a token's heads of one kind (0: q, 1: k, 2: v), kRows heads
// a step.  c, z: the rotation.
template <int D, int kind>
MOE_DEV void append_heads(const KvAppendArgs &a, int t, int from, int to, const uint64_t (&c)[4],
                          const uint64_t (&z)[4], Place place) {
    constexpr int kLanes = D / 16, kRows = 32 / kLanes, NG = D / 32;
    if (from >= to) return;
    const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
    const int heads = kind == 0 ? a.q_heads : a.pool.hkv, ps = a.pool.ps;
    const uint16_t *base = (kind == 0   ? a.q + (size_t)t * a.q_stride
                            : kind == 1 ? a.k + (size_t)t * a.k_stride
                                        : a.v + (size_t)t * a.v_stride) + 8 * l;
    // lanes past the last head repeat it and write nothing
    auto row = [&](int step) { return base + min(step * kRows + sub, heads - 1) * D; };
    const uint16_t *w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    uint64_t w0[4], w1[4];
    if (kind < 2 && w) {
        unpack8(*reinterpret_cast<const uint4 *>(w + 8 * l), w0);
        unpack8(*reinterpret_cast<const uint4 *>(w + D / 2 + 8 * l), w1);
    }
    const uint64_t minus1 = pair(-1.0f, -1.0f);
    // the rows of this step and of the next kAhead, so that enough bytes are on their way
    constexpr int kAhead = 2;
    uint4 nx[kAhead], ny[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const uint16_t *src = row(min(from + i, to - 1));
        nx[i] = *reinterpret_cast<const uint4 *>(src);
        ny[i] = *reinterpret_cast<const uint4 *>(src + D / 2);
    }
#pragma unroll 1
    for (int step = from; step < to; ++step) {
        const int head = step * kRows + sub;
        uint64_t x2[4], y2[4];
        unpack8(nx[0], x2);
        unpack8(ny[0], y2);
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) {
            nx[i] = nx[i + 1];
            ny[i] = ny[i + 1];
        }
        if (step + kAhead < to) {
            const uint16_t *src = row(step + kAhead);
            nx[kAhead - 1] = *reinterpret_cast<const uint4 *>(src);
            ny[kAhead - 1] = *reinterpret_cast<const uint4 *>(src + D / 2);
        }
        if (kind < 2 && w) {
            // sum of squares of the row, in the documented order
            uint64_t s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = add2(prod2(x2[j], x2[j]), prod2(y2[j], y2[j]));
            const float2 f = both(add2(add2(s[0], s[2]), add2(s[1], s[3])));
            float sum = __fadd_rn(f.x, f.y);
#pragma unroll
            for (int m = 1; m < kLanes; m <<= 1)
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, m));
            const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / D), a.eps)));
            const uint64_t r2 = pair(r, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x2[j] = mul2(mul2(x2[j], r2), w0[j]);
                y2[j] = mul2(mul2(y2[j], r2), w1[j]);
            }
        }
        if (kind < 2 && a.cos) {
            if (!a.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) turn2(x2[j], y2[j], c[j], z[j], minus1);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 cx = both(c[j / 2]), zx = both(z[j / 2]);
                    const float2 cy = both(c[2 + j / 2]), zy = both(z[2 + j / 2]);
                    x2[j] = turn1(x2[j], j & 1 ? cx.y : cx.x, j & 1 ? zx.y : zx.x);
                    y2[j] = turn1(y2[j], j & 1 ? cy.y : cy.x, j & 1 ? zy.y : zy.x);
                }
            }
        }
        if (kind == 0) {
            if (head < heads) {
                uint16_t *dst = a.q_out + ((size_t)t * heads + head) * D + 8 * l;
                *reinterpret_cast<uint4 *>(dst) = pack8(x2);
                *reinterpret_cast<uint4 *>(dst + D / 2) = pack8(y2);
            }
            continue;
        }
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = both(x2[j]), g = both(y2[j]);
            x[2 * j] = f.x, x[2 * j + 1] = f.y;
            y[2 * j] = g.x, y[2 * j + 1] = g.y;
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
        const bool mine = head < heads && place.page;
        if (limited && mine) kv_report(a.err, MOE_KV4_DEVERR_RANGE);
        // the lane's eighth of its two groups G and NG/2 + G
        const int tq = l & 3, G = l >> 2, G2 = NG / 2 + G;
        uint32_t first, second;
        if (kind == 1) {
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
        uint8_t *blk = place.page + (size_t)head * a.pool.block;
        uint8_t *codes = blk + (kind == 1 ? 0 : ps * (D / 2)) + place.slot * (D / 2);
        uint16_t *sc =
            reinterpret_cast<uint16_t *>(blk + ps * D) + (kind == 1 ? 0 : ps * NG) + place.slot * NG;
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

template <int D>
__global__ void __launch_bounds__(256, 3) kv4_append_kernel(const KvAppendArgs a) {
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    pdl_wait();
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int t = warp / a.split, share = warp - t * a.split;
    if (t >= a.batch.tokens) return;
    // the token's steps of kRows heads: q, then k, then v; this warp's part of them
    const int nq = (a.q_heads + kRows - 1) / kRows, nk = (a.pool.hkv + kRows - 1) / kRows;
    const int steps = nq + 2 * nk;
    const int from = steps * share / a.split, to = steps * (share + 1) / a.split;
    Place place{nullptr, 0};
    int at = 0;
    bool owned = true;  // by a request
    if (to > nq || (a.cos && !a.positions)) {
        const int b = kv_request_of(a.batch.cu_q, a.batch.requests, t);
        at = kv_index_of(a.batch, b, t, owned);
        // of no request, or more new tokens than the sequence's length: not stored
        if (to > nq && at >= 0) {
            const int page =
                kv_page_of(a.batch, a.pool, b, at, lane == 0 && to == steps ? a.err : nullptr);
            if (page >= 0) place = Place{kv_block(a.pool, page, 0), at % a.pool.ps};
        }
    }
    uint64_t c[4] = {}, z[4] = {};
    if (a.cos && from < nq + nk) {
        int pos = a.positions ? a.positions[t] : at;
        if (pos < 0 || pos >= a.max_pos) {
            if (lane == 0 && share == 0 && (owned || a.positions))
                kv_report(a.err, MOE_KV4_DEVERR_POSITION);
            pos = min(max(pos, 0), a.max_pos - 1);
        }
        const float *cs = a.cos + (size_t)pos * (D / 2), *sn = a.sin + (size_t)pos * (D / 2);
        if (!a.interleaved) {
            load8(cs + 8 * l, c);
            load8(sn + 8 * l, z);
        } else {
            // pairs of the row's first half, then of its second
            const ulonglong2 c0 = *reinterpret_cast<const ulonglong2 *>(cs + 4 * l);
            const ulonglong2 c1 = *reinterpret_cast<const ulonglong2 *>(cs + D / 4 + 4 * l);
            const ulonglong2 z0 = *reinterpret_cast<const ulonglong2 *>(sn + 4 * l);
            const ulonglong2 z1 = *reinterpret_cast<const ulonglong2 *>(sn + D / 4 + 4 * l);
            c[0] = c0.x, c[1] = c0.y, c[2] = c1.x, c[3] = c1.y;
            z[0] = z0.x, z[1] = z0.y, z[2] = z1.x, z[3] = z1.y;
        }
    }
    append_heads<D, 0>(a, t, from, min(to, nq), c, z, place);
    append_heads<D, 1>(a, t, max(from, nq) - nq, min(to, nq + nk) - nq, c, z, place);
    append_heads<D, 2>(a, t, max(from, nq + nk) - nq - nk, to - nq - nk, c, z, place);
}

// One row (token, head, K or V) per D/16 lanes, as in the append.  6800 tokens of 8 heads
// of 128: 10.4 us for 36 MB, half the copy's rate: a lane has one row, so one dependent
// round trip (lengths, page id, codes) and, for V, loads of two bytes.
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
    bool owned;
    const int at = kv_index_of(a.batch, b, t, owned);
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
