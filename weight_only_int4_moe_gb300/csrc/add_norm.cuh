// The residual's addition and the root-mean-square norm of each row (moe_add_norm):
//   h = x + residual,  y = h * (1 / sqrt(sum h^2 / H + eps)) * weight,
// y rounded to the output's type and, where wanted, to e4m3 codes with one scale a row.
//
// Bound by memory: x and the residual are read once, the row stays in registers, and h, y
// and the codes are written once.  A block has one row; its threads hold vectors of eight
// elements.  Where rows begin elsewhere than at multiples of 16 bytes, but all matrices' rows
// at the same place between two (contiguous rows of any length), the vectors lie on that grid
// and the two at the row's ends are moved by elements (ENDS; single elements throughout took
// 90 instructions each: 4096 rows of 4095 70 us, now 36).  What is left goes by single elements.
//
// Measured: 8192 rows of 7168 bf16 with a residual 75 us, 6.2 TB/s of the 6.8 that a copy reaches;
// 2048 rows of 4096, fp32 into a bf16 stream, with codes 16.5 us (5.6 TB/s); one row 2.9 us.
//
// An 8-bit code is decided by y to the last bit wherever y / scale lies next to the middle
// of two codes, and y by the sum of squares.  So the sum should not depend on how a row is
// cut into threads: it is held as a number and its rounding error (two-sum: the error of an
// addition is itself an fp32 number), some 45 bits in all, and rounded once at the end.  One
// row in a million or fewer then has another sum than 64 bits give (measured: 1 of 3.1 million
// rows of 4096), where the sum lies next to the middle of two fp32 numbers.
#pragma once

#include <cfloat>

#include "layer.cuh"

namespace moe {

namespace {

// A sum as hi + lo, hi = fl(hi + lo).
struct Sum2 {
    float hi, lo;
};
// a + b = s + e exactly (Knuth's two-sum).
MOE_DEV void two_sum(float a, float b, float &s, float &e) {
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}
MOE_DEV void add_square(Sum2 &t, float h) {
    const float q = __fmul_rn(h, h);
    float s, e;
    two_sum(t.hi, q, s, e);
    t.hi = s;
    t.lo = __fadd_rn(t.lo, __fadd_rn(e, __fmaf_rn(h, h, -q)));
}
MOE_DEV Sum2 join(Sum2 a, Sum2 b) {
    float s, e;
    two_sum(a.hi, b.hi, s, e);
    e = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
    // not renormalised: lo stays far below hi, and the order of joining does not matter
    // beyond lo's own rounding
    return Sum2{s, e};
}

// VEC consecutive elements of a type as they lie in memory.
template <int TYPE, int VEC>
struct Elems {
    static constexpr int kWords = TYPE == MOE_T_F32 ? VEC : VEC / 2;
    uint32_t w[kWords ? kWords : 1];

    MOE_DEV void load(const void *p, int64_t i) {
        if constexpr (VEC == 1) {
            if constexpr (TYPE == MOE_T_F32)
                w[0] = reinterpret_cast<const uint32_t *>(p)[i];
            else
                w[0] = reinterpret_cast<const uint16_t *>(p)[i];
        } else {
            const uint4 *q = reinterpret_cast<const uint4 *>(
                reinterpret_cast<const char *>(p) + i * (TYPE == MOE_T_F32 ? 4 : 2));
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k) {
                const uint4 v = q[k];
                w[4 * k] = v.x;
                w[4 * k + 1] = v.y;
                w[4 * k + 2] = v.z;
                w[4 * k + 3] = v.w;
            }
        }
    }
    MOE_DEV void store(void *p, int64_t i) const {
        if constexpr (VEC == 1) {
            if constexpr (TYPE == MOE_T_F32)
                reinterpret_cast<uint32_t *>(p)[i] = w[0];
            else
                reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)w[0];
        } else {
            uint4 *q = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(p) +
                                                 i * (TYPE == MOE_T_F32 ? 4 : 2));
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k)
                q[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
    }
    // The elements that exist of a vector that begins at element p of a row of H (from `row`).
    MOE_DEV void load_part(const void *row, int p, int H) {
        zero();
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (p + j >= 0 && p + j < H) {
                if constexpr (TYPE == MOE_T_F32)
                    w[j] = reinterpret_cast<const uint32_t *>(row)[p + j];
                else
                    w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[p + j] << (j & 1) * 16;
            }
    }
    MOE_DEV void store_part(void *row, int p, int H) const {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (p + j >= 0 && p + j < H) {
                if constexpr (TYPE == MOE_T_F32)
                    reinterpret_cast<uint32_t *>(row)[p + j] = w[j];
                else
                    reinterpret_cast<uint16_t *>(row)[p + j] = (uint16_t)(w[j / 2] >> (j & 1) * 16);
            }
    }
    MOE_DEV void zero() {
#pragma unroll
        for (int k = 0; k < (kWords ? kWords : 1); ++k) w[k] = 0u;
    }
    MOE_DEV float get(int j) const {
        if constexpr (TYPE == MOE_T_F32) return __uint_as_float(w[j]);
        const uint32_t v = (j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu;
        if constexpr (TYPE == MOE_T_BF16) return __uint_as_float(v << 16);
        return __half2float(__ushort_as_half((uint16_t)v));
    }
    // Rounds f to the type.
    MOE_DEV void set(const float (&f)[VEC]) {
        if constexpr (TYPE == MOE_T_F32) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[j] = __float_as_uint(f[j]);
        } else if constexpr (VEC == 1) {
            w[0] = to_bits16(f[0], TYPE);
        } else {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                if constexpr (TYPE == MOE_T_BF16)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(w[j])
                        : "f"(f[2 * j + 1]), "f"(f[2 * j]));
                else
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                        : "=r"(w[j])
                        : "f"(f[2 * j + 1]), "f"(f[2 * j]));
            }
        }
    }
};

// Element access of a thread's vectors: those that begin at element p of a row of H.
template <int VEC, bool ENDS>
struct Span {
    int H;
    MOE_DEV bool any(int p) const { return ENDS ? p < H && p + VEC > 0 : p < H; }
    MOE_DEV bool whole(int p) const { return !ENDS || (p >= 0 && p + VEC <= H); }
    template <int TYPE>
    MOE_DEV void load(Elems<TYPE, VEC> &e, const void *base, int64_t row, int p) const {
        if (whole(p))
            e.load(base, row + p);
        else
            e.load_part(reinterpret_cast<const char *>(base) + row * (TYPE == MOE_T_F32 ? 4 : 2), p, H);
    }
    template <int TYPE>
    MOE_DEV void store(const Elems<TYPE, VEC> &e, void *base, int64_t row, int p) const {
        if (whole(p))
            e.store(base, row + p);
        else
            e.store_part(reinterpret_cast<char *>(base) + row * (TYPE == MOE_T_F32 ? 4 : 2), p, H);
    }
    MOE_DEV void store_as(const MatOut &o, int64_t row, int p, const float (&f)[VEC]) const {
        if (o.type == MOE_T_F32) {
            Elems<MOE_T_F32, VEC> v;
            v.set(f);
            store(v, o.p, row, p);
        } else if (o.type == MOE_T_BF16) {
            Elems<MOE_T_BF16, VEC> v;
            v.set(f);
            store(v, o.p, row, p);
        } else {
            Elems<MOE_T_F16, VEC> v;
            v.set(f);
            store(v, o.p, row, p);
        }
    }
};

// A thread's weights: two-byte ones as they lie in memory so that
// all are asked for before any is waited for; fp32 ones are loaded where they are used.
template <int VEC, int NV, bool ENDS>
struct Weights {
    Elems<MOE_T_BF16, VEC> w[NV];
    MOE_DEV void load(const AddNormArgs &a, int T, int tid, int first) {
        if (a.weight_type == MOE_T_F32) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int p = first + (i * T + tid) * VEC;
            const Span<VEC, ENDS> span{a.hidden};
            if (!span.any(p)) continue;
            if (span.whole(p) && first == 0)
                w[i].load(a.weight, p);
            else if constexpr (ENDS)  // (weights begin at a multiple of 16 bytes, rows do not)
                w[i].load_part(a.weight, p, a.hidden);
        }
    }
    MOE_DEV void get(const AddNormArgs &a, int i, int p, float (&f)[VEC]) const {
        if (a.weight_type == MOE_T_F32) {
            Elems<MOE_T_F32, VEC> v;
            if constexpr (ENDS)
                v.load_part(a.weight, p, a.hidden);
            else
                v.load(a.weight, p);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = v.get(j);
        } else if (a.weight_type == MOE_T_BF16) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = w[i].get(j);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const uint32_t v = (j & 1) ? w[i].w[j / 2] >> 16 : w[i].w[j / 2] & 0xFFFFu;
                f[j] = __half2float(__ushort_as_half((uint16_t)v));
            }
        }
    }
};

MOE_DEV uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr int kNone = -1;  // no residual

// TX, TS: types of x and of the residual; VEC: elements of a load; NV: loads of a thread;
// MAX: threads of a block at most; ENDS: the row's ends may lie inside a vector.
template <int TX, int TS, int VEC, int NV, int MAX, bool ENDS>
__global__ void __launch_bounds__(MAX, 1024 / MAX) add_norm_kernel(const AddNormArgs a) {
    __shared__ float part_hi[32], part_lo[32], part_max[32];
    __shared__ double part_d[32];
    const int row = blockIdx.x, tid = threadIdx.x, T = blockDim.x, lane = tid & 31;
    const int warps = T >> 5, H = a.hidden;
    constexpr bool kAdd = TS != kNone;
    constexpr int kHeld = kAdd ? TS : TX;  // h has this type exactly: it is kept as it lies in memory
    const Span<VEC, ENDS> span{H};
    // the first vector's element: at or in front of the row's first
    const int first = ENDS ? -((row & 7) * a.stride8 & 7) : 0;
    pdl_wait();
    pdl_launch_dependents();

    Elems<kHeld, VEC> h[NV];
    Weights<VEC, NV, ENDS> weights;
    constexpr bool kEarly = NV <= 8;  // else they would not fit beside the row
    if constexpr (kAdd) {
        Elems<TX, VEC> x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int p = first + (i * T + tid) * VEC;
            if (span.any(p)) {
                span.load(x[i], a.x.p, row * a.x.stride, p);
                span.load(h[i], a.residual.p, row * a.residual.stride, p);
            }
        }
        if (kEarly && a.weight) weights.load(a, T, tid, first);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int p = first + (i * T + tid) * VEC;
            if (span.any(p)) {
                float f[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) f[j] = __fadd_rn(x[i].get(j), h[i].get(j));
                h[i].set(f);
                if (a.residual_out.p)
                    span.store(h[i], a.residual_out.p, row * a.residual_out.stride, p);
            } else {
                h[i].zero();
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int p = first + (i * T + tid) * VEC;
            h[i].zero();
            if (span.any(p)) span.load(h[i], a.x.p, row * a.x.stride, p);
        }
        if (kEarly && a.weight) weights.load(a, T, tid, first);
    }

    Sum2 t{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) add_square(t, h[i].get(j));
#pragma unroll
    for (int o = 16; o; o >>= 1)
        t = join(t, Sum2{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
    if (warps > 1) {
        if (lane == 0) {
            part_hi[tid >> 5] = t.hi;
            part_lo[tid >> 5] = t.lo;
        }
        __syncthreads();
        t = lane < warps ? Sum2{part_hi[lane], part_lo[lane]} : Sum2{0.0f, 0.0f};
#pragma unroll
        for (int o = 16; o; o >>= 1)
            t = join(t, Sum2{__shfl_xor_sync(0xffffffffu, t.hi, o),
                             __shfl_xor_sync(0xffffffffu, t.lo, o)});
    }
    // the compensation of an infinite or NaN sum is NaN: the sum itself counts then
    const float total = fabsf(t.hi) <= FLT_MAX ? __fadd_rn(t.hi, t.lo) : t.hi;
    float q, up = 1.0f;
    if (!(total < 1e37f) || (total < 1e-30f && a.eps < 1e-24f)) {
        // squares beyond fp32, or below it with nothing added to them
        double d = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) d += (double)h[i].get(j) * (double)h[i].get(j);
#pragma unroll
        for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (warps > 1) {
            if (lane == 0) part_d[tid >> 5] = d;
            __syncthreads();
            d = lane < warps ? part_d[lane] : 0.0;
#pragma unroll
            for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        }
        // 1 / sqrt is a normal number for root mean squares between 2^-100 and 2^100.  Rows
        // beyond them come to the middle by a power of two, which costs their elements nothing
        // that y could show.
        const double ms = d / H + (double)a.eps;
        if (ms > 0.0 && ms < 0x1p-200) up = 0x1p96f;
        if (ms > 0x1p200 && ms < INFINITY) up = 0x1p-32f;
        q = (float)(1.0 / (sqrt(ms) * (double)up));
    } else {
        q = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(total, a.inv_hidden), a.eps)));
    }

    if (!kEarly && a.weight) weights.load(a, T, tid, first);
    float top = 0.0f, y[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int p = first + (i * T + tid) * VEC;
        if (span.any(p)) {
            float f[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = 1.0f;
            if (a.weight) weights.get(a, i, p, f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                y[i][j] = __fmul_rn(__fmul_rn(__fmul_rn(h[i].get(j), up), q), f[j]);
                // (NaN is not counted, nor what lies beyond the row's ends: 0 times an
                // infinite 1 / sqrt is NaN)
                top = fmaxf(top, fabsf(y[i][j]));
            }
            if (a.out.p) span.store_as(a.out, row * a.out.stride, p, y[i]);
        }
    }
    if (!a.codes) return;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (warps > 1) {
        if (lane == 0) part_max[tid >> 5] = top;
        __syncthreads();
        top = lane < warps ? part_max[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const float scale = fmaxf(__fmul_rn(top, 1.0f / 448.0f), 0x1p-100f);
    const float inv = __frcp_rn(scale);
    if (tid == 0) a.scales[row] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int p = first + (i * T + tid) * VEC;
        if (!span.any(p)) continue;
        uint8_t *c = a.codes + row * a.codes_stride + p;
        if constexpr (VEC == 1) {
            *c = (uint8_t)e4m3x2(__fmul_rn(y[i][0], inv), 0.0f);
        } else {
            uint32_t v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                v[k] = e4m3x2(__fmul_rn(y[i][4 * k], inv), __fmul_rn(y[i][4 * k + 1], inv)) |
                       (uint32_t)e4m3x2(__fmul_rn(y[i][4 * k + 2], inv),
                                        __fmul_rn(y[i][4 * k + 3], inv))
                           << 16;
            if (span.whole(p)) {
                *reinterpret_cast<uint2 *>(c) = make_uint2(v[0], v[1]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (p + j >= 0 && p + j < H) c[j] = (uint8_t)(v[j / 4] >> (j & 3) * 8);
            }
        }
    }
}

template <int TX, int TS, int VEC, int NV, int MAX, bool ENDS>
cudaError_t launch(const AddNormArgs &a, cudaStream_t s) {
    const int per = VEC * NV, n = a.hidden + (ENDS ? VEC - 1 : 0), T = ((n + per - 1) / per + 31) / 32 * 32;
    auto c = pdl_config((unsigned)a.rows, (unsigned)T, 0, s);
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return cudaLaunchKernelEx(&c, add_norm_kernel<TX, TS, VEC, NV, MAX, ENDS>, a);
}

// Rows beyond 8192 take 1024 threads with 64 registers each, which spill 32 to 376 bytes a thread
// (2048 rows of 16384 with a residual: bf16 47 us, 5.8 TB/s; fp32 96, 4.9 TB/s; bf16 with codes
// 53), as do the kernels without vectors (up to 684).
//
// Loads of a thread: one for short rows and for a row or two an SM, where the latency counts;
// else four, so that more rows are in flight on an SM (8192 rows of 7168 bf16 with a residual:
// 132 us with one, 91 with two, 75 with four).
template <int TX, int TS>
cudaError_t by_size(const AddNormArgs &a, Grid grid, int sms, cudaStream_t s) {
    // fp32 rows take twice the registers: two loads (8192 rows of 7168 fp32 with an fp32 residual
    // 117 us, four 157)
    constexpr bool kWide = TS != kNone && (TX == MOE_T_F32 || TS == MOE_T_F32);
    constexpr int kLoads = kWide ? 2 : 4, kMost = 8192 / (8 * kLoads);
    if (grid == Grid::kVectors) {
        if (a.hidden <= 8192) {
            if (a.hidden <= 1024 || a.rows <= 2 * sms) return launch<TX, TS, 8, 1, 1024, false>(a, s);
            return launch<TX, TS, 8, kLoads, kMost, false>(a, s);
        }
        return launch<TX, TS, 8, 4, 1024, false>(a, s);
    }
    if (grid == Grid::kEnds) {
        if (a.hidden <= 8184) return launch<TX, TS, 8, kLoads, kMost, true>(a, s);
        if (a.hidden <= 32760) return launch<TX, TS, 8, 4, 1024, true>(a, s);
    }
    if (a.hidden <= 4096) return launch<TX, TS, 1, 8, 512, false>(a, s);
    return launch<TX, TS, 1, 32, 1024, false>(a, s);
}

}  // namespace

template <int TX>
cudaError_t add_norm_of(const AddNormArgs &a, Grid grid, int sms, cudaStream_t s) {
    if (!a.residual.p) return by_size<TX, kNone>(a, grid, sms, s);
    if (a.residual.type == MOE_T_BF16) return by_size<TX, MOE_T_BF16>(a, grid, sms, s);
    if (a.residual.type == MOE_T_F16) return by_size<TX, MOE_T_F16>(a, grid, sms, s);
    return by_size<TX, MOE_T_F32>(a, grid, sms, s);
}

}  // namespace moe
