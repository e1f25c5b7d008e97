// Matrix products with an epilogue (moe_linear):
//   out[m][n] = act(sum_k x[m][k] w[n][k] * sx[m] * sw[n] + bias[n]) * gate[m][n] + residual[m][n]
//
// The tensor cores' M side (the 128 lanes of tensor memory) takes rows of w, their N side TN
// rows of x: a few tokens then waste little, and a warp's 32 lanes hold 32 neighbouring
// columns of one output row, so that the epilogue reads and writes whole sectors without a
// detour through shared memory, whatever the matrices' strides.  Both operands come by TMA in
// stages of 128 bytes of k (64 two-byte elements or 128 codes); what lies outside a matrix is
// filled with zeros.
//
// Two kernels.  Where the tiles fill the GPU, linear_pair_kernel: two blocks work on one tile
// of 256 rows of w by TN of x, each holding its half of either operand, and walk over tiles
// with the sums in two buffers, so that the epilogue of a tile runs under the products of the
// next.  Otherwise linear_split_kernel: one tile of 128 by TN a cluster, whose blocks share the
// tile's k and add their parts up through distributed shared memory, in the order of the
// blocks: no workspace, and the same bits every time.
//
// What bounds them: a few tokens the weights' way from HBM (1 x 7168 x 7168 18.2 us, 5.7 TB/s of
// the 6.7 that a copy reaches), sizes between a block's stages (a 128-byte row is one request of
// the copy engine: about 100 GB/s a block; 256 x 2048 x 7168 with SiLU and gate 14.5 us, 13.2 with
// the weights in L2), large products the tensor cores (8192 x 7168 x 7168 427 us, 1970 TFLOP/s,
// where cuBLAS reached 1929 at 8192^3; in a row the power cap, 500 us).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "layer.cuh"

namespace moe {

namespace {

constexpr int kRowsW = 128;                 // rows of w of a block's tile
constexpr int kLine = 128;                  // bytes of k of a stage
constexpr int kBytesW = kRowsW * kLine;
constexpr int kThreads = 320;               // warps 0-7 epilogue, 8 copies, 9 products
constexpr int kEpilogue = 8;                // warps
constexpr int kPairThreads = 576;           // of a pair's block: warps 0-15 epilogue, 16 copies, 17 products
constexpr int kPairEpilogue = 16;
constexpr int kMaxSmem = 227 * 1024 - 1024; // of a block, beside its few static bytes
constexpr int kHalfSmem = 110 * 1024;       // where two lie on an SM

MOE_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
MOE_DEV uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
MOE_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of another block's shared memory.
MOE_DEV uint32_t map_to(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
MOE_DEV float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
MOE_DEV void prefetch_2d(const void *tmap, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(c0), "r"(c1)
                 : "memory");
}
MOE_DEV void arrive_at(uint32_t addr) {  // (an address of map_to)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Instruction descriptor: fp32 sums, both operands K-major, m rows by n.
MOE_DEV uint32_t idesc_of(int type, uint32_t m, uint32_t n) {
    const uint32_t f = type == MOE_T_BF16 ? 1u : 0u;  // kind::f16: 1 bf16, 0 f16; f8f6f4: 0 e4m3
    return (1u << 4) | (f << 7) | (f << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// The four products of a stage (32 bytes of k each) from one elected thread, then the commit
// that hands the stage back: to this block, or for a pair to both.
#define MOE_MMA4(GROUP, KIND, COMMIT)                                                      \
    asm volatile(                                                                          \
        "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t.reg .b16 both;\n\t" \
        "setp.ne.b32 p, %4, 0;\n\t"                                                        \
        "setp.eq.b32 t, %4, %4;\n\t"                                                       \
        "mov.b16 both, 3;\n\t"                                                             \
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"               \
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"               \
        "elect.sync _|e, 0xffffffff;\n\t"                                                  \
        "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t"      \
        "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a1, b1, %3, t;\n\t"      \
        "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a2, b2, %3, t;\n\t"      \
        "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a3, b3, %3, t;\n\t"      \
        "@e tcgen05.commit.cta_group::" GROUP COMMIT ";\n\t}" ::"r"(d),                    \
        "l"(wd), "l"(xd), "r"(idesc), "r"(accumulate), "r"(bar)                            \
        : "memory")
#define MOE_COMMIT_ONE ".mbarrier::arrive::one.shared::cluster.b64 [%5]"
#define MOE_COMMIT_BOTH ".mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], both"
template <bool CODES, bool PAIR>
MOE_DEV void mma_stage(uint32_t d, uint64_t wd, uint64_t xd, uint32_t idesc, uint32_t accumulate,
                       uint32_t bar) {
    if constexpr (PAIR && CODES)
        MOE_MMA4("2", "f8f6f4", MOE_COMMIT_BOTH);
    else if constexpr (PAIR)
        MOE_MMA4("2", "f16", MOE_COMMIT_BOTH);
    else if constexpr (CODES)
        MOE_MMA4("1", "f8f6f4", MOE_COMMIT_ONE);
    else
        MOE_MMA4("1", "f16", MOE_COMMIT_ONE);
}
#undef MOE_MMA4
#undef MOE_COMMIT_ONE
#undef MOE_COMMIT_BOTH
// Arrives on both blocks' barrier once the products issued so far are done.
MOE_DEV void commit_both(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 both;\n\tmov.b16 both, 3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], both;\n\t}" ::"r"(bar)
        : "memory");
}

// Tensor memory -> registers: issued, and waited for with the registers as operands, so that
// no use of them moves ahead of the wait.
template <int C>
struct Cols {
    static_assert(C == 16, "columns of a load");
    uint32_t r[C];
    MOE_DEV void issue(uint32_t taddr) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
            "%11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr)
            : "memory");
    }
    MOE_DEV void wait() {
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                       "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                       "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                     :
                     : "memory");
    }
};

// 16 columns of n sums that lie `apart` columns from each other, added up.
MOE_DEV void add_sums(uint32_t taddr, int n, int apart, float (&v)[16]) {
    Cols<16> acc;
    acc.issue(taddr);
    acc.wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(acc.r[j]);
#pragma unroll 1
    for (int i = 1; i < n; ++i) {
        acc.issue(taddr + i * apart);
        acc.wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(acc.r[j]);
    }
}

// --------------------------------------------------------------- epilogue --
MOE_DEV float from_bits16(uint32_t v, int type) {
    return type == MOE_T_BF16 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half((uint16_t)v));
}

template <int C>
MOE_DEV void activate(int act, float (&v)[C]) {
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = v[j] / (1.0f + expf(-v[j]));
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = 0.5f * v[j] * (1.0f + erff(v[j] * 0.7071067811865476f));
    }
}

// Two neighbouring columns of a matrix in eight rows two apart, as they lie in memory.
struct Pairs {
    uint32_t r[16];
    MOE_DEV void load(const MatIn &s, int m, int n, int cols) {
        const int64_t at = (int64_t)m * s.stride + n;
        if (s.type == MOE_T_F32) {
            const float *p = reinterpret_cast<const float *>(s.p) + at;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint2 v = 2 * q < cols ? *reinterpret_cast<const uint2 *>(p + 2 * q * s.stride)
                                             : make_uint2(0u, 0u);
                r[2 * q] = v.x, r[2 * q + 1] = v.y;
            }
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(s.p) + at;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                r[q] = 2 * q < cols ? *reinterpret_cast<const uint32_t *>(p + 2 * q * s.stride) : 0u;
        }
    }
    MOE_DEV void get(int type, float (&f)[16]) const {
        if (type == MOE_T_F32) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
        } else if (type == MOE_T_BF16) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                f[2 * q] = __uint_as_float(r[q] << 16);
                f[2 * q + 1] = __uint_as_float(r[q] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&r[q]));
                f[2 * q] = v.x;
                f[2 * q + 1] = v.y;
            }
        }
    }
};

// The block's part of a tile: 128 columns from n0 by `rows` output rows from m0, in the sums at
// `tmem`.  A warp takes the lanes it can reach and every WARPS / 4-th run of 16 rows.  A lane has one
// column of the sums; lanes 2i and 2i + 1 trade, so that either has both columns of every other
// row, and a row takes half the accesses.  (Each lane with its own column, two bytes an access,
// 34 instructions an element made the epilogue the bound: 8192 x 7168 from K = 512 with a
// residual 143 us.)  The gate and the residual of a run are asked for DEPTH runs ahead, the
// first ones before the sums are complete (begin).
template <int DEPTH, int WARPS>
struct TileOut {
    static constexpr int C = 16, kStep = WARPS / 4 * C;
    Pairs gate[DEPTH], residual[DEPTH];
    int m0, rows, n, c;
    float sw, bias;

    // the rows of run `at` that this lane has after the trade: at + odd, at + odd + 2, ...
    MOE_DEV void load(const LinearArgs &a, int at, Pairs &g, Pairs &r) {
        const int odd = n & 1, cols = rows - at - odd;
        if (!a.vec2 || n >= a.N || cols <= 0) return;
        if (a.gate.p) g.load(a.gate, m0 + at + odd, n - odd, cols);
        if (a.residual.p) r.load(a.residual, m0 + at + odd, n - odd, cols);
    }
    MOE_DEV void begin(const LinearArgs &a, int m0_, int n0, int rows_, int w, int lane) {
        m0 = m0_, rows = rows_, n = n0 + (w & 3) * 32 + lane, c = (w >> 2) * C;
        sw = n < a.N && a.w_scale ? a.w_scale[n] : 1.0f;
        bias = n < a.N && a.bias ? a.bias[n] : 0.0f;
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(a, c + kStep * d, gate[d], residual[d]);
    }
    // From n sums, `apart` columns from each other.
    MOE_DEV void run(const LinearArgs &a, uint32_t tmem, int w, int n_sums, int apart) {
        const uint32_t lanes = tmem + ((uint32_t)(w & 3) << 21);
#pragma unroll 1
        while (c < rows) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (c >= rows) break;
                float v[C];
                add_sums(lanes + c, n_sums, apart, v);
                emit(a, v, gate[d], residual[d]);
            }
        }
    }
    // The next run, from its sums.
    MOE_DEV void emit(const LinearArgs &a, float (&v)[C], Pairs &g, Pairs &r) {
        if (a.x_scale) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (c + j < rows) v[j] *= a.x_scale[m0 + c + j];
        }
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = v[j] * sw + bias;
        activate<C>(a.activation, v);
        if (a.vec2)
            pairs(a, v, g, r);
        else if (n < a.N)
            singles(a, v);
        load(a, c + kStep * DEPTH, g, r);
        c += kStep;
    }
    MOE_DEV void pairs(const LinearArgs &a, float (&v)[C], const Pairs &g, const Pairs &r) {
        const int odd = n & 1, cols = rows - c - odd;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? v[2 * q] : v[2 * q + 1], 1);
            v[2 * q] = odd ? other : v[2 * q];
            v[2 * q + 1] = odd ? v[2 * q + 1] : other;
        }
        if (n >= a.N) return;
        float f[C];
        if (a.gate.p) {
            g.get(a.gate.type, f);
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] *= f[j];
        }
        if (a.residual.p) {
            r.get(a.residual.type, f);
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] += f[j];
        }
        const int64_t at = (int64_t)(m0 + c + odd) * a.out.stride + (n - odd);
        if (a.out.type == MOE_T_F32) {
            float *p = reinterpret_cast<float *>(a.out.p) + at;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (2 * q < cols)
                    *reinterpret_cast<float2 *>(p + 2 * q * a.out.stride) = make_float2(v[2 * q], v[2 * q + 1]);
        } else {
            uint16_t *p = reinterpret_cast<uint16_t *>(a.out.p) + at;
            uint32_t b[8];
            if (a.out.type == MOE_T_BF16) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[q]) : "f"(v[2 * q + 1]), "f"(v[2 * q]));
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(b[q]) : "f"(v[2 * q + 1]), "f"(v[2 * q]));
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (2 * q < cols) *reinterpret_cast<uint32_t *>(p + 2 * q * a.out.stride) = b[q];
        }
    }
    // Matrices whose neighbours are not one access: the lane's own column.
    static MOE_DEV void own(const MatIn &s, int m, int n, int cols, float (&f)[C]) {
        const int64_t at = (int64_t)m * s.stride + n;
        if (s.type == MOE_T_F32) {
            const float *p = reinterpret_cast<const float *>(s.p) + at;
#pragma unroll
            for (int j = 0; j < C; ++j) f[j] = j < cols ? p[j * s.stride] : 0.0f;
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(s.p) + at;
            uint16_t b[C];
#pragma unroll
            for (int j = 0; j < C; ++j) b[j] = j < cols ? p[j * s.stride] : (uint16_t)0;
#pragma unroll
            for (int j = 0; j < C; ++j) f[j] = from_bits16(b[j], s.type);
        }
    }
    MOE_DEV void singles(const LinearArgs &a, float (&v)[C]) {
        const int m = m0 + c, cols = rows - c;
        float f[C];
        if (a.gate.p) {
            own(a.gate, m, n, cols, f);
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] *= f[j];
        }
        if (a.residual.p) {
            own(a.residual, m, n, cols, f);
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] += f[j];
        }
        const int64_t at = (int64_t)m * a.out.stride + n;
        if (a.out.type == MOE_T_F32) {
            float *p = reinterpret_cast<float *>(a.out.p) + at;
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (j < cols) p[j * a.out.stride] = v[j];
        } else {
            uint16_t *p = reinterpret_cast<uint16_t *>(a.out.p) + at;
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (j < cols) p[j * a.out.stride] = to_bits16(v[j], a.out.type);
        }
    }
};

// Asks for a tile's gate and residual in L2 (one thread a row).
MOE_DEV void row_lines(const MatIn &s, int m, int n0, int N) {
    const int size = s.type == MOE_T_F32 ? 4 : 2;
    const char *p = reinterpret_cast<const char *>(s.p) + ((int64_t)m * s.stride + n0) * size;
    for (int i = 0; i < min(kRowsW, N - n0) * size; i += 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
}
MOE_DEV void tile_lines(const LinearArgs &a, int m0, int n0, int rows, int tid) {
    const int m = m0 + tid;
    if (tid >= rows || m >= a.M || n0 >= a.N) return;
    if (a.gate.p) row_lines(a.gate, m, n0, a.N);
    if (a.residual.p) row_lines(a.residual, m, n0, a.N);
}

// Four neighbours of a row, n..n+3 (those below N exist), as they lie in memory: nothing waits
// for a load before its values are used.
struct Quad {
    uint32_t r[4];
    MOE_DEV void load(const MatIn &s, bool vec, int m, int n, int N) {
        const int64_t at = (int64_t)m * s.stride + n;
        if (s.type == MOE_T_F32) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(s.p) + at;
            if (vec && n + 3 < N) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p);
                r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = n + j < N ? p[j] : 0u;
            }
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(s.p) + at;
            if (vec && n + 3 < N) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                r[0] = v.x, r[1] = v.y;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = n + j < N ? p[j] : 0u;
            }
        }
    }
    MOE_DEV void get(int type, bool vec, int n, int N, float (&f)[4]) const {
        if (type == MOE_T_F32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(r[j]);
        } else if (vec && n + 3 < N) {
            f[0] = from_bits16(r[0] & 0xFFFFu, type), f[1] = from_bits16(r[0] >> 16, type);
            f[2] = from_bits16(r[1] & 0xFFFFu, type), f[3] = from_bits16(r[1] >> 16, type);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = from_bits16(r[j], type);
        }
    }
};

MOE_DEV void quad_out(const LinearArgs &a, int m, int n, float (&v)[4], const float (&sw)[4],
                      const float (&bias)[4], const Quad &gate, const Quad &residual, float sx) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * sx * sw[j] + bias[j];
    activate<4>(a.activation, v);
    if (a.gate.p) {
        gate.get(a.gate.type, a.vec_gate, n, a.N, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= f[j];
    }
    if (a.residual.p) {
        residual.get(a.residual.type, a.vec_residual, n, a.N, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += f[j];
    }
    const int64_t at = (int64_t)m * a.out.stride + n;
    if (a.out.type == MOE_T_F32) {
        float *p = reinterpret_cast<float *>(a.out.p) + at;
        if (a.vec_out && n + 3 < a.N) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < a.N) p[j] = v[j];
        }
    } else {
        uint16_t *p = reinterpret_cast<uint16_t *>(a.out.p) + at;
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = to_bits16(v[j], a.out.type);
        if (a.vec_out && n + 3 < a.N) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < a.N) p[j] = (uint16_t)b[j];
        }
    }
}

// ----------------------------------------------------- one tile a cluster --
// How a product is cut: rows of x of a tile (a multiple of 16), blocks that share a tile's k,
// stages of a block, and sums that the lines of k go to in turn.
struct Cut {
    int tn, split, stages, sums;
    int stage_bytes() const { return kBytesW + tn * kLine; }
    int smem() const { return stages * stage_bytes() + 1024; }  // (stages begin at multiples of 1024)
};
constexpr int kMaxStages = 12, kMaxSplit = 8;

// Lines of k that one sum in tensor memory takes where the result stays fp32.  The tensor cores
// cut a sum's last place with every instruction, 4 a line: the error of a random product,
// relative to it, measured 1.7e-8 an instruction (K = 7168 in one sum 7.9e-6).  So longer products
// go to several sums, which are added up in fp32.  16-bit results show it from kLongLines on
// (2048 instructions, 3e-5: a 15th of fp16's half step).
constexpr int kExactLines = 12, kLongLines = 512;

// (Bounded as blocks of 12 warps: 10 lie on an SM's four parts as 3, 3, 2 and 2, so that of two
// blocks with 96 registers a thread the second would not fit.)
template <bool CODES>
__global__ void __launch_bounds__(384, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap, const LinearArgs a, const int tn,
                        const int n_stages, const int n_sums) {
    extern __shared__ uint8_t dyn[];
    __shared__ alignas(8) uint64_t bars[2 * kMaxStages + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), S = cluster_size();
    const int n0 = (int)(blockIdx.x / S) * kRowsW, m0 = (int)blockIdx.y * tn;
    const uint32_t stage_bytes = kBytesW + tn * kLine;
    const uint32_t stages = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxStages, done = full + 16 * kMaxStages;
    const int all = tn * n_sums;
    const uint32_t cols = all <= 32 ? 32 : all <= 64 ? 64 : all <= 128 ? 128 : all <= 256 ? 256 : 512;
    constexpr int kElems = CODES ? kLine : kLine / 2;
    const int kb = (a.K + kElems - 1) / kElems;
    const int kb0 = (int)((int64_t)kb * rank / S), kb1 = (int)((int64_t)kb * (rank + 1) / S);

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2 * kMaxStages + 1; ++i) mbar_init(full + 8 * i, 1);
        mbar_fence_init();
    }
    // The first lines of w come to L2 while the previous kernel ends.
    if (w == 8 && lane < n_stages && kb0 + lane < kb1) prefetch_2d(&wmap, (kb0 + lane) * kElems, n0);
    // Tensor memory is taken behind the previous kernel, whose blocks may still want theirs, and
    // before the next one may start.  Kernels of other streams do not want it beside this one: two
    // blocks of this kernel take 256 columns each where they share an SM, and for any other kernel
    // that has tensor memory an SM has too few registers left (the expert GEMMs 768 x 80, the
    // prefill attention 896 x 72) or too little shared memory (pairs).  A block that waited for
    // columns while its cluster waits for it could wait for ever.
    pdl_wait();
    if (w == 9) {
        tmem_alloc(smem_u32(&tmem_slot), cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_launch_dependents();

    if (w == 8) {
        if (lane == 0) {
            Ring r(n_stages);
            int issued = 0;
            for (int k = kb0; k < kb1; ++k, r.next()) {
                if (!mbar_wait(empty + 8 * r.idx, r.ph ^ 1, &abort_flag, a.err)) break;
                const uint32_t bar = full + 8 * r.idx, s = stages + r.idx * stage_bytes;
                mbar_arrive_expect_tx(bar, stage_bytes);
                if (!(kDebugBounds && issued == a.skip_line && blockIdx.x == 0 && blockIdx.y == 0))
                    tma_load_2d(s, &wmap, k * kElems, n0, bar);
                tma_load_2d(s + kBytesW, &xmap, k * kElems, m0, bar);
                ++issued;
            }
            if (*(volatile int *)&abort_flag) {
                // the copies in flight end before the block does
                volatile int none = 0;
                Ring q(n_stages);
                for (int i = 0; i < issued; ++i, q.next())
                    if (i >= issued - n_stages) mbar_wait(full + 8 * q.idx, q.ph, &none, a.err);
            }
        }
        __syncwarp();
    } else if (w == 9) {
        const uint32_t idesc = idesc_of(a.type, 128, tn);
        Ring r(n_stages);
        int sum = 0;
        for (int k = kb0; k < kb1; ++k, r.next(), sum = sum + 1 == n_sums ? 0 : sum + 1) {
            if (__any_sync(0xffffffffu, !mbar_wait(full + 8 * r.idx, r.ph, &abort_flag, a.err))) break;
            tc_fence_after();
            const uint32_t s = stages + r.idx * stage_bytes;
            mma_stage<CODES, false>(tmem + sum * tn, smem_desc_sw128(s), smem_desc_sw128(s + kBytesW),
                                    idesc, k >= kb0 + n_sums, empty + 8 * r.idx);
        }
        tc_commit_elect(done);
        if (__any_sync(0xffffffffu, *(volatile int *)&abort_flag)) {
            // products in flight end before the tensor memory is given back
            volatile int none = 0;
            mbar_wait(done, 0, &none, a.err);
        }
    }
    // The sums are complete, and with them every copy has been used.
    __syncwarp();
    const int rows = min(tn, a.M - m0);  // output rows of the tile
    if (S == 1) {
        if (w < kEpilogue) {
            TileOut<1, kEpilogue> out;
            out.begin(a, m0, n0, rows, w, lane);
            mbar_wait(done, 0, &abort_flag, a.err);
            __syncwarp();
            tc_fence_after();
            out.run(a, tmem, w, n_sums, tn);
        }
    } else {
        // Of the output a warp will take a row of its block's share at a time, a lane four
        // columns.  A row's gate and residual are asked for while the row before it is worked
        // on, the first row's before the sums are complete.
        const int c0 = rows * (int)rank / (int)S, c1 = rows * (int)(rank + 1) / (int)S;
        const int n = n0 + 4 * lane;
        Quad gate, residual;
        const auto ask = [&](int c) {
            if (c >= c1) return;
            if (a.gate.p) gate.load(a.gate, a.vec_gate, m0 + c, n, a.N);
            if (a.residual.p) residual.load(a.residual, a.vec_residual, m0 + c, n, a.N);
        };
        if (w < kEpilogue) {
            ask(c0 + w);
            mbar_wait(done, 0, &abort_flag, a.err);
            __syncwarp();
            tc_fence_after();
        }
        // parts[m][n]: 128 fp32 numbers for each output row
        if (w < kEpilogue) {
            const uint32_t at = stages + 4 * (uint32_t)((w & 3) * 32 + lane);
            const uint32_t lanes = tmem + ((uint32_t)(w & 3) << 21);
#pragma unroll 1
            for (int c = (w >> 2) * 16; c < rows; c += 32) {
                float v[16];
                add_sums(lanes + c, n_sums, tn, v);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + (c + j) * 512), "f"(v[j]) : "memory");
            }
        }
        __syncwarp();
        cluster_sync();
        if (w < kEpilogue) {
            float sw[4], bias[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sw[j] = a.w_scale && n + j < a.N ? a.w_scale[n + j] : 1.0f;
                bias[j] = a.bias && n + j < a.N ? a.bias[n + j] : 0.0f;
            }
#pragma unroll 1
            for (int c = c0 + w; c < c1; c += kEpilogue) {
                const int m = m0 + c;
                const float sx = a.x_scale ? a.x_scale[m] : 1.0f;
                const uint32_t at = stages + c * 512 + 16 * lane;
                float4 p[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < S) p[q] = ld_cluster4(map_to(at, q));
                const Quad g = gate, r = residual;
                ask(c + kEpilogue);
                float v[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
#pragma unroll
                for (int q = 1; q < 8; ++q)
                    if (q < S) v[0] += p[q].x, v[1] += p[q].y, v[2] += p[q].z, v[3] += p[q].w;
                quad_out(a, m, n, v, sw, bias, g, r, sx);
            }
        }
        __syncwarp();
        cluster_sync();  // the others have read this block's parts
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 9) tmem_dealloc(tmem, cols);
}

// ------------------------------------------------ two blocks, many tiles --
// Lines of k up to which a tile's epilogue takes longer than its products: there the next tile's
// gate and residual are asked for in L2 (8192 x 7168 from K = 512 with a residual 90 -> 82 us).
// Behind longer products they come in time by themselves, and asking costs 1 %.
constexpr int kShortLines = 18;

template <int TN>
struct Pair {
    static constexpr int kStage = kBytesW + TN / 2 * kLine;  // of one block
    static constexpr int kStages = TN == 256 ? 6 : 8;
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr uint32_t kCols = 2 * TN;
    static constexpr int kBars = 2 * kStages + 5;  // full, empty, sums full, sums empty, end
};

// A pair's copy: its bytes are counted by the first block's barrier (an address of map_to).
MOE_DEV void tma_load_pair(uint32_t dst, const void *tmap, int32_t c0, int32_t c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Tiles are taken in bands of kBand along x's rows, so that what runs at the same time shares
// rows of both operands in L2.
constexpr int kBand = 8;
MOE_DEV void tile_at(int t, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int band = t / (kBand * tiles_n), r = t - band * kBand * tiles_n;
    const int high = min(kBand, tiles_m - band * kBand);
    tn = r / high;
    tm = band * kBand + r - tn * high;
}

// LONG: a tile's k in parts of kExactLines, each a sum of its own in one of the two buffers, that
// the epilogue adds up in registers.
template <int TN, bool CODES, bool LONG>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap xmap, const LinearArgs a) {
    using T = Pair<TN>;
    extern __shared__ uint8_t dyn[];
    __shared__ alignas(8) uint64_t bars[T::kBars];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;
    const int tiles_n = (a.N + 2 * kRowsW - 1) / (2 * kRowsW), tiles_m = (a.M + TN - 1) / TN;
    const int tiles = tiles_m * tiles_n;
    const uint32_t stages = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * T::kStages;
    const uint32_t sums_full = full + 16 * T::kStages, sums_empty = sums_full + 16;
    const uint32_t end = sums_empty + 16;
    constexpr int kElems = CODES ? kLine : kLine / 2;
    const int kb = (a.K + kElems - 1) / kElems, part = LONG ? kExactLines : kb;

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < T::kBars; ++i)
            mbar_init(full + 8 * i, i == 2 * T::kStages + 2 || i == 2 * T::kStages + 3 ? 2 * kPairEpilogue : 1);
        mbar_fence_init();
    }
    pdl_wait();
    if (w == kPairEpilogue + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_slot)),
                     "r"(T::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other block's barriers are there
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_launch_dependents();

    if (w == kPairEpilogue) {
        if (lane == 0) {
            const uint32_t full0 = map_to(full, 0);
            Ring r(T::kStages);
            int issued = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                int tm, tn;
                tile_at(t, tiles_m, tiles_n, tm, tn);
                const int n0 = tn * 2 * kRowsW + (int)rank * kRowsW, m0 = tm * TN + (int)rank * (TN / 2);
                for (int k = 0; k < kb; ++k, r.next()) {
                    ok = mbar_wait(empty + 8 * r.idx, r.ph ^ 1, &abort_flag, a.err);
                    if (!ok) break;
                    const uint32_t s = stages + r.idx * T::kStage;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * r.idx, 2 * T::kStage);
                    if (!(kDebugBounds && issued == a.skip_line && blockIdx.x == 0))
                        tma_load_pair(s, &wmap, k * kElems, n0, full0 + 8 * r.idx);
                    tma_load_pair(s + kBytesW, &xmap, k * kElems, m0, full0 + 8 * r.idx);
                    ++issued;
                }
            }
            if (rank == 0 && *(volatile int *)&abort_flag) {
                // the copies in flight, of both blocks, end before the blocks do
                volatile int none = 0;
                Ring q(T::kStages);
                for (int i = 0; i < issued; ++i, q.next())
                    if (i >= issued - T::kStages) mbar_wait(full + 8 * q.idx, q.ph, &none, a.err);
            }
        }
        __syncwarp();
    } else if (w == kPairEpilogue + 1) {
        if (rank == 0) {
            const uint32_t idesc = idesc_of(a.type, 256, TN);
            Ring r(T::kStages), acc(2);
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step)
                for (int k0 = 0; k0 < kb && ok; k0 += part, acc.next()) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(sums_empty + 8 * acc.idx, acc.ph ^ 1, &abort_flag, a.err));
                    tc_fence_after();
                    for (int k = k0; k < min(kb, k0 + part) && ok; ++k, r.next()) {
                        ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * r.idx, r.ph, &abort_flag, a.err));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t s = stages + r.idx * T::kStage;
                        mma_stage<CODES, true>(tmem + acc.idx * TN, smem_desc_sw128(s),
                                               smem_desc_sw128(s + kBytesW), idesc, k > k0,
                                               empty + 8 * r.idx);
                    }
                    if (ok) commit_both(sums_full + 8 * acc.idx);
                }
            if (!ok) {
                // products in flight end before the tensor memory is given back
                volatile int none = 0;
                commit_both(end);
                mbar_wait(end, 0, &none, a.err);
                __syncwarp();
            }
        }
    } else {
        const uint32_t empty0 = map_to(sums_empty, 0);
        Ring acc(2);
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            int tm, tn;
            tile_at(t, tiles_m, tiles_n, tm, tn);
            TileOut<1, kPairEpilogue> out;
            out.begin(a, tm * TN, tn * 2 * kRowsW + (int)rank * kRowsW, min(TN, a.M - tm * TN), w, lane);
            if (kb <= kShortLines && t + step < tiles) {
                int next_m, next_n;
                tile_at(t + step, tiles_m, tiles_n, next_m, next_n);
                tile_lines(a, next_m * TN, next_n * 2 * kRowsW + (int)rank * kRowsW, TN, tid);
            }
            constexpr int kRuns = LONG ? TN / (kPairEpilogue * 4) : 1;  // of 16 rows, of a warp
            float total[kRuns][16];
            for (int k0 = 0; k0 < kb && ok; k0 += part, acc.next()) {
                ok = __all_sync(0xffffffffu, mbar_wait(sums_full + 8 * acc.idx, acc.ph, &abort_flag, a.err));
                if (!ok) break;
                tc_fence_after();
                const uint32_t sums = tmem + acc.idx * TN;
                if constexpr (LONG) {
                    const uint32_t lanes = sums + ((uint32_t)(w & 3) << 21) + (w >> 2) * 16;
#pragma unroll
                    for (int i = 0; i < kRuns; ++i) {
                        Cols<16> v;
                        v.issue(lanes + i * kPairEpilogue * 4);
                        v.wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            total[i][j] = (k0 ? total[i][j] : 0.0f) + __uint_as_float(v.r[j]);
                    }
                } else {
                    out.run(a, sums, w, 1, 0);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(empty0 + 8 * acc.idx);
            }
            if constexpr (LONG) {
#pragma unroll
                for (int i = 0; i < kRuns; ++i)
                    if (ok && out.c < out.rows) out.emit(a, total[i], out.gate[0], out.residual[0]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (w == kPairEpilogue + 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(T::kCols)
                     : "memory");
}

// ------------------------------------------------------------------- host --
// Tensor map over rows of k, one 128-byte line of a row wide, box_rows high.
bool rows_map(CUtensorMap *m, const void *p, int64_t stride, int rows, int K, int type, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int size = type == MOE_T_E4M3 ? 1 : 2;
    // (the stride of a single row is not used, but has to be a valid one)
    cuuint64_t pitch = rows > 1 ? (cuuint64_t)stride * size : ((cuuint64_t)K * size + 15) / 16 * 16;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint32_t box[2] = {(cuuint32_t)(kLine / size), (cuuint32_t)box_rows};
    cuuint32_t step[2] = {1, 1};
    const CUtensorMapDataType t = type == MOE_T_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                  : type == MOE_T_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto encode = [&] {
        return fn(m, t, 2, const_cast<void *>(p), dims, &pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // The driver wants a current context, which a thread does not have before its first call
    // that needs one; this one may be its first.
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// What a launch needs to know of the operands.
struct Operands {
    const void *x, *w;
    int64_t x_stride, w_stride;
    int sms;
};

// Allows a kernel its shared memory, once a device; *n: clusters that fit on it at once (for
// a kernel of pairs).
template <typename K>
cudaError_t prepare(K kernel, int smem, std::atomic<int> *known, int *n, int pair_grid) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && known[dev] > 0) {
        *n = known[dev];
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    *n = 1;
    if (pair_grid) {
        cudaLaunchConfig_t c{};
        c.gridDim = dim3((unsigned)pair_grid);
        c.blockDim = dim3(kPairThreads);
        c.dynamicSmemBytes = smem;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 2;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        c.numAttrs = 1;
        c.attrs = &at;
        e = cudaOccupancyMaxActiveClusters(n, kernel, &c);
        if (e != cudaSuccess) return e;
        if (*n < 1) return cudaErrorLaunchOutOfResources;
    }
    if (dev >= 0 && dev < 64) known[dev] = *n;
    return cudaSuccess;
}

thread_local int last_kernel = 0;  // MOE_LINEAR_*

template <int TN, bool CODES, bool LONG>
cudaError_t launch_pair(const LinearArgs &a, const Operands &o, cudaStream_t s) {
    using T = Pair<TN>;
    static std::atomic<int> known[64];
    int pairs;
    cudaError_t e = prepare(linear_pair_kernel<TN, CODES, LONG>, T::kSmem, known, &pairs, o.sms / 2 * 2);
    if (e != cudaSuccess) return e;
    CUtensorMap wmap, xmap;
    if (!rows_map(&wmap, o.w, o.w_stride, a.N, a.K, a.type, kRowsW) ||
        !rows_map(&xmap, o.x, o.x_stride, a.M, a.K, a.type, TN / 2))
        return cudaErrorNotSupported;
    const int64_t tiles = (int64_t)((a.N + 2 * kRowsW - 1) / (2 * kRowsW)) * ((a.M + TN - 1) / TN);
    auto c = pdl_config((unsigned)(2 * (tiles < pairs ? tiles : pairs)), kPairThreads, T::kSmem, s);
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    e = cudaLaunchKernelEx(&c, linear_pair_kernel<TN, CODES, LONG>, wmap, xmap, a);
    if (e == cudaSuccess)
        last_kernel = TN == 256 ? MOE_LINEAR_PAIRS_256 : LONG ? MOE_LINEAR_PAIRS_128_SUMS : MOE_LINEAR_PAIRS_128;
    return e;
}

template <bool CODES>
cudaError_t launch_split(const LinearArgs &a, const Operands &o, const Cut &cut, cudaStream_t s) {
    // (the parts lie where the stages were)
    if (cut.stages < 2 || cut.tn * cut.sums > 512 || cut.tn * kRowsW * 4 > cut.stages * cut.stage_bytes()) return cudaErrorInvalidValue;
    static std::atomic<int> known[64];
    int one;
    cudaError_t e = prepare(linear_split_kernel<CODES>, kMaxSmem, known, &one, 0);
    if (e != cudaSuccess) return e;
    CUtensorMap wmap, xmap;
    if (!rows_map(&wmap, o.w, o.w_stride, a.N, a.K, a.type, kRowsW) ||
        !rows_map(&xmap, o.x, o.x_stride, a.M, a.K, a.type, cut.tn))
        return cudaErrorNotSupported;
    auto c = pdl_config(1, kThreads, (size_t)cut.smem(), s);
    c.gridDim = dim3((unsigned)((a.N + kRowsW - 1) / kRowsW * cut.split),
                     (unsigned)((a.M + cut.tn - 1) / cut.tn));
    cudaLaunchAttribute at[2] = {};
    c.numAttrs = 1 + pdl_attr(at[0]);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cut.split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    e = cudaLaunchKernelEx(&c, linear_split_kernel<CODES>, wmap, xmap, a, cut.tn, cut.stages, cut.sums);
    if (e == cudaSuccess) last_kernel = MOE_LINEAR_SPLIT;
    return e;
}

// sums: wanted (tensor memory bounds them)
Cut make_cut(int tn, int split, int per_sm, int sums) {
    Cut c{tn, split, 0, std::min(sums, 512 / per_sm / tn)};
    c.stages = ((per_sm == 1 ? kMaxSmem : kHalfSmem) - 1024) / c.stage_bytes();
    if (c.stages > kMaxStages) c.stages = kMaxStages;
    return c;
}

// Times in us, from what was measured of the kernels' parts:
//  - A block takes a line of k in 170 ns and 0.65 ns for each of its tn rows of x (its waits,
//    and the copies' requests, one a row); two blocks on an SM get a row in 0.93 ns.  Rows that
//    do not begin at multiples of 128 bytes take two requests a line: 1.4 times that.
//  - w comes from HBM once, at 6.6 TB/s; less by up to 6 % with the blocks that an SM could hold
//    more.
//  - An epilogue of two warps a quarter of the lanes takes 0.55 us for 32 rows (twice that where
//    columns do not go in pairs); parts cost 1.2 us for the two cluster barriers, 0.12 us for
//    32 rows to write them and 0.25 us for 8 rows of a block's share to add them up.
//  - 2 us for the launch and the first lines; lines take 1.8 us more where blocks share an SM;
//    every further block of an SM adds 1.5 us for its own and its epilogue.
//  - A pair takes a line in 0.33 us (256 rows of x) or 0.22 us (128), under which runs the
//    epilogue of the tile before, 6.2 and 3.7 us; 3 us for its start.
struct Size {
    int M, N, kb, sms;
    // columns go in pairs; rows begin at multiples of 128 bytes; no sum takes more than kExactLines
    bool even, lined, exact;
    double hbm() const { return ((double)N + M) * kb * kLine / 6.6e6; }
    bool operator==(const Size &o) const {
        return M == o.M && N == o.N && kb == o.kb && sms == o.sms && even == o.even && lined == o.lined &&
               exact == o.exact;
    }
};

double split_time(const Size &z, const Cut &c, int per_sm) {
    const double blocks = (double)((z.N + kRowsW - 1) / kRowsW) * ((z.M + c.tn - 1) / c.tn) * c.split;
    const double waves = std::ceil(blocks / ((double)z.sms * per_sm));
    double line = 170 + 0.65 * c.tn;
    if (per_sm == 2) line = std::max(line, 0.93 * (kRowsW + c.tn) * std::min(2.0, std::ceil(blocks / z.sms)));
    if (!z.lined) line *= 1.4;
    const double rows = std::min(c.tn, z.M);
    const double out = c.split == 1 ? (z.even ? 0.55 : 1.1) * std::ceil(rows / 32)
                                    : 1.2 + 0.12 * std::ceil(rows / 32) +
                                          0.25 * std::ceil(rows / c.split / 8);
    const double idle = std::max(0.0, 1 - blocks / (z.sms * per_sm));
    const double lines = waves * line * std::ceil((double)z.kb / c.split) / 1000 + 1.8 * (per_sm - 1);
    return 2 + std::max(z.hbm() * (1 + 0.06 * idle), lines) + out +
           (waves - 1) * (1.5 + out);
}

double pair_time(const Size &z, int tn) {
    const double tiles = (double)((z.N + 2 * kRowsW - 1) / (2 * kRowsW)) * ((z.M + tn - 1) / tn);
    const double work = z.kb * (tn == 256 ? 0.33 : 0.22), out = (tn == 256 ? 6.2 : 3.7) * (z.even ? 1 : 2);
    return 3 + std::max(z.hbm(), std::ceil(tiles / (z.sms / 2)) * std::max(work, out)) +
           std::min(work, out);
}

// The fastest cut by that; fits[per_sm - 1][split]: blocks that run at the same time (clusters
// lie inside a group of SMs, so not all of them can be used).
Cut best_cut(const Size &z, const int (&fits)[2][kMaxSplit + 1], double *time) {
    Cut best{};
    *time = 1e30;
    const int whole = (z.M + 15) / 16 * 16;
    for (int tn : {16, 32, 48, 64, 96, 128, whole}) {
        if (tn > whole || tn > 128) continue;
        const int64_t tiles = (int64_t)((z.N + kRowsW - 1) / kRowsW) * ((z.M + tn - 1) / tn);
        if ((z.M + tn - 1) / tn > 65535) continue;  // (the grid's second dimension)
        for (int split = 1; split <= kMaxSplit && split * 3 <= std::max(z.kb, 3); ++split)
            for (int per_sm = 1; per_sm <= 2; ++per_sm) {
                const int sums = z.exact ? ((z.kb + split - 1) / split + kExactLines - 1) / kExactLines : 1;
                const Cut c = make_cut(tn, split, per_sm, sums);
                if (c.sums < sums) continue;
                if (c.stages < 3 || (split > 1 && tiles * split > fits[per_sm - 1][split])) continue;
                const double t = split_time(z, c, per_sm);
                if (t < *time) {
                    *time = t;
                    best = c;
                }
            }
    }
    return best;
}

// fits of best_cut on the current device, asked once.  Of two blocks an SM the clusters of one
// are counted twice, which is never too many (asked for them, the runtime says one an SM, but
// two do run).
template <bool CODES>
cudaError_t cluster_room(int (&fits)[2][kMaxSplit + 1]) {
    static std::atomic<int> known[64][kMaxSplit + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < 64;
    for (int split = 1; split <= kMaxSplit; ++split) {
        int n = keep ? known[dev][split].load() : 0;
        if (n <= 0) {
            cudaLaunchConfig_t c{};
            c.gridDim = dim3((unsigned)split);
            c.blockDim = dim3(kThreads);
            c.dynamicSmemBytes = (size_t)kMaxSmem;
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = (unsigned)split;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            c.numAttrs = 1;
            c.attrs = &at;
            e = cudaFuncSetAttribute(linear_split_kernel<CODES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kMaxSmem);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, linear_split_kernel<CODES>, &c);
            if (e != cudaSuccess) return e;
            if (keep) known[dev][split] = n;
        }
        fits[0][split] = n * split;
        fits[1][split] = 2 * n * split;
    }
    return cudaSuccess;
}

// What a product's sizes decide: the kernel (pair: rows of x of a pair's tile, or 0) and its cut.
struct Plan {
    Size z;
    int pair;
    Cut cut;
};

Plan make_plan(const Size &z, const int (&fits)[2][kMaxSplit + 1]) {
    double split;
    Plan p{z, 0, best_cut(z, fits, &split)};
    const double wide = z.exact && z.kb > kExactLines ? 1e30 : pair_time(z, 256), half = pair_time(z, 128);
    if (split > std::min(wide, half)) p.pair = half < wide ? 128 : 256;
    return p;
}

// The plan of a size, worked out once (5 us) and kept by each thread for its last sizes.
template <bool CODES>
cudaError_t plan_of(const Size &z, Plan *plan) {
    static thread_local Plan kept[64];
    uint32_t h = (uint32_t)z.M * 2654435761u ^ (uint32_t)z.N * 2246822519u ^ (uint32_t)z.kb * 3266489917u;
    h ^= (uint32_t)(z.even + 2 * z.lined + 4 * z.exact) * 668265263u;
    Plan &k = kept[(h ^ h >> 15) % 64];
    if (!(k.z == z)) {
        int fits[2][kMaxSplit + 1];
        const cudaError_t e = cluster_room<CODES>(fits);
        if (e != cudaSuccess) return e;
        k = make_plan(z, fits);
    }
    *plan = k;
    return cudaSuccess;
}

template <bool CODES>
cudaError_t by_size(const LinearArgs &a, const Operands &o, cudaStream_t s) {
    const int size = CODES ? 1 : 2;
    const auto at_lines = [&](const void *p, int64_t stride, int rows) {
        return (uintptr_t)p % kLine == 0 && (rows == 1 || stride * size % kLine == 0);
    };
    const int kb = (a.K * size + kLine - 1) / kLine;
    const Size z{a.M, a.N, kb, o.sms, a.vec2,
                 at_lines(o.x, o.x_stride, a.M) && at_lines(o.w, o.w_stride, a.N),
                 a.out.type == MOE_T_F32 || kb > kLongLines};
    Plan p;
    const cudaError_t e = plan_of<CODES>(z, &p);
    if (e != cudaSuccess) return e;
    if (p.pair == 256) return launch_pair<256, CODES, false>(a, o, s);
    if (p.pair == 128)
        return z.exact && z.kb > kExactLines ? launch_pair<128, CODES, true>(a, o, s)
                                             : launch_pair<128, CODES, false>(a, o, s);
    return launch_split<CODES>(a, o, p.cut, s);
}

// `count` neighbours of a row may be one access.
bool together(const void *p, int64_t stride, int type, int rows, int count) {
    const int bytes = (type == MOE_T_F32 ? 4 : 2) * count;
    return !p || (((uintptr_t)p % bytes) == 0 && (rows == 1 || stride % count == 0));
}

}  // namespace

int linear_last_kernel() { return last_kernel; }

cudaError_t launch_linear(LinearArgs a, const void *x, int64_t x_stride, const void *w,
                          int64_t w_stride, int sms, cudaStream_t s) {
    a.vec_gate = together(a.gate.p, a.gate.stride, a.gate.type, a.M, 4);
    a.vec_residual = together(a.residual.p, a.residual.stride, a.residual.type, a.M, 4);
    a.vec_out = together(a.out.p, a.out.stride, a.out.type, a.M, 4);
    a.vec2 = a.N % 2 == 0 && together(a.gate.p, a.gate.stride, a.gate.type, a.M, 2) &&
             together(a.residual.p, a.residual.stride, a.residual.type, a.M, 2) &&
             together(a.out.p, a.out.stride, a.out.type, a.M, 2);
    const Operands o{x, w, x_stride, w_stride, sms};
    return a.type == MOE_T_E4M3 ? by_size<true>(a, o, s) : by_size<false>(a, o, s);
}

}  // namespace moe
