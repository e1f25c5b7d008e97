// Matrix products with an epilogue (moe_linear):
//   out[m][n] = act(sum_k x[m][k] w[n][k] * sx[m] * sw[n] + bias[n]) * gate[m][n] + residual[m][n]
//
// The tensor cores' M side (128 lanes of tensor memory) takes 128 rows of w, their N side TN
// rows of x: a few tokens then waste little, and a warp's 32 lanes hold 32 neighbouring
// columns of one output row, so that the epilogue reads and writes whole sectors without a
// detour through shared memory, whatever the matrices' strides.  Both operands come by TMA in
// stages of 128 bytes of k (64 two-byte elements or 128 codes); what lies outside a matrix is
// filled with zeros.
//
// One tile a cluster.  Where there are too few tiles for the GPU, the blocks of a cluster share
// a tile's k and add their parts up through distributed shared memory, in the order of the
// blocks: no workspace, and the same bits every time.
#include <atomic>

#include "layer.cuh"

namespace moe {

namespace {

constexpr int kRowsW = 128;                 // rows of w of a tile
constexpr int kLine = 128;                  // bytes of k of a stage
constexpr int kBytesW = kRowsW * kLine;
constexpr int kThreads = 192;               // warps 0-3 epilogue, 4 copies, 5 products

template <int TN>
struct Tile {
    static constexpr int kStage = kBytesW + TN * kLine;
    static constexpr int kStages = TN >= 128 ? 4 : 5;
    static constexpr int kSmem = kStages * kStage + 1024;  // (stages begin at multiples of 1024)
    static constexpr uint32_t kCols = TN < 32 ? 32 : TN;   // of tensor memory
    static_assert(TN * kRowsW * 4 <= kStages * kStage, "the parts lie where the stages were");
};

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
MOE_DEV float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Instruction descriptor: fp32 sums, both operands K-major, 128 rows by n.
MOE_DEV uint32_t idesc_of(int type, uint32_t n) {
    const uint32_t f = type == MOE_T_BF16 ? 1u : 0u;  // kind::f16: 1 bf16, 0 f16; f8f6f4: 0 e4m3
    return (1u << 4) | (f << 7) | (f << 10) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// The four products of a stage (32 bytes of k each) from one elected thread, then the commit
// that hands the stage back.
template <bool CODES>
MOE_DEV void mma_stage(uint32_t d, uint64_t wd, uint64_t xd, uint32_t idesc, uint32_t accumulate,
                       uint32_t bar) {
#define MOE_MMA4(KIND)                                                                     \
    asm volatile(                                                                          \
        "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                \
        "setp.ne.b32 p, %4, 0;\n\t"                                                        \
        "setp.eq.b32 t, %4, %4;\n\t"                                                       \
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"               \
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"               \
        "elect.sync _|e, 0xffffffff;\n\t"                                                  \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], %1, %2, %3, p;\n\t"              \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a1, b1, %3, t;\n\t"              \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a2, b2, %3, t;\n\t"              \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a3, b3, %3, t;\n\t"              \
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"( \
            d),                                                                            \
        "l"(wd), "l"(xd), "r"(idesc), "r"(accumulate), "r"(bar)                            \
        : "memory")
    if constexpr (CODES)
        MOE_MMA4("f8f6f4");
    else
        MOE_MMA4("f16");
#undef MOE_MMA4
}

template <int C>
MOE_DEV void load_column(const MatIn &s, int m, int n, int cols, float (&f)[C]) {
    const int64_t at = (int64_t)m * s.stride + n;
    if (s.type == MOE_T_F32) {
        const float *p = reinterpret_cast<const float *>(s.p) + at;
#pragma unroll
        for (int j = 0; j < C; ++j) f[j] = j < cols ? p[j * s.stride] : 0.0f;
    } else {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(s.p) + at;
        uint16_t v[C];
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = j < cols ? p[j * s.stride] : (uint16_t)0;
        if (s.type == MOE_T_BF16) {
#pragma unroll
            for (int j = 0; j < C; ++j) f[j] = __uint_as_float((uint32_t)v[j] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) f[j] = __half2float(__ushort_as_half(v[j]));
        }
    }
}

// The epilogue of C neighbouring output rows m.. (cols of them exist) in column n.
template <int C>
MOE_DEV void finish(const LinearArgs &a, int m, int n, int cols, float (&v)[C], float sw,
                    float bias) {
    if (a.x_scale) {
#pragma unroll
        for (int j = 0; j < C; ++j)
            if (j < cols) v[j] *= a.x_scale[m + j];
    }
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = v[j] * sw + bias;
    if (a.activation == MOE_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
    } else if (a.activation == MOE_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = v[j] / (1.0f + expf(-v[j]));
    } else if (a.activation == MOE_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = 0.5f * v[j] * (1.0f + erff(v[j] * 0.7071067811865476f));
    }
    float f[C];
    if (a.gate.p) {
        load_column<C>(a.gate, m, n, cols, f);
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] *= f[j];
    }
    if (a.residual.p) {
        load_column<C>(a.residual, m, n, cols, f);
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

template <int TN, bool CODES>
__global__ void __launch_bounds__(kThreads)
    linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                  const LinearArgs a) {
    using T = Tile<TN>;
    extern __shared__ uint8_t dyn[];
    __shared__ alignas(8) uint64_t bars[2 * T::kStages + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), S = cluster_size();
    const int n0 = (int)(blockIdx.x / S) * kRowsW, m0 = (int)blockIdx.y * TN;
    const uint32_t stages = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * T::kStages, done = full + 16 * T::kStages;
    constexpr int kElems = CODES ? kLine : kLine / 2;
    const int kb = (a.K + kElems - 1) / kElems;
    const int kb0 = (int)((int64_t)kb * rank / S), kb1 = (int)((int64_t)kb * (rank + 1) / S);

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2 * T::kStages + 1; ++i) mbar_init(full + 8 * i, 1);
        mbar_fence_init();
    }
    if (w == 5) {
        tmem_alloc(smem_u32(&tmem_slot), T::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (w == 4) {
        if (lane == 0) {
            Ring r(T::kStages);
            int issued = 0;
            for (int k = kb0; k < kb1; ++k, r.next()) {
                if (!mbar_wait(empty + 8 * r.idx, r.ph ^ 1, &abort_flag, a.err)) break;
                const uint32_t bar = full + 8 * r.idx, s = stages + r.idx * T::kStage;
                mbar_arrive_expect_tx(bar, T::kStage);
                tma_load_2d(s, &wmap, k * kElems, n0, bar);
                tma_load_2d(s + kBytesW, &xmap, k * kElems, m0, bar);
                ++issued;
            }
            if (*(volatile int *)&abort_flag) {
                // the copies in flight end before the block does
                volatile int none = 0;
                Ring q(T::kStages);
                for (int i = 0; i < issued; ++i, q.next())
                    if (i >= issued - T::kStages) mbar_wait(full + 8 * q.idx, q.ph, &none, a.err);
            }
        }
        __syncwarp();
    } else if (w == 5) {
        const uint32_t idesc = idesc_of(a.type, TN);
        Ring r(T::kStages);
        for (int k = kb0; k < kb1; ++k, r.next()) {
            if (__any_sync(0xffffffffu, !mbar_wait(full + 8 * r.idx, r.ph, &abort_flag, a.err))) break;
            tc_fence_after();
            const uint32_t s = stages + r.idx * T::kStage;
            mma_stage<CODES>(tmem, smem_desc_sw128(s), smem_desc_sw128(s + kBytesW), idesc,
                             k > kb0, empty + 8 * r.idx);
        }
        tc_commit_elect(done);  // also after giving up: products in flight end first
    }
    // The sums are complete, and with them every copy has been used.
    __syncwarp();
    if (w < 4) {
        mbar_wait(done, 0, &abort_flag, a.err);
        __syncwarp();
        tc_fence_after();
    }
    const int n = n0 + (w & 3) * 32 + lane;
    const bool mine = w < 4 && n < a.N;
    const float sw = mine && a.w_scale ? a.w_scale[n] : 1.0f;
    const float bias = mine && a.bias ? a.bias[n] : 0.0f;
    const int rows = min(TN, a.M - m0);  // output rows of the tile
    const uint32_t quarter = tmem + ((uint32_t)(w & 3) << 21);
    if (S == 1) {
        if (w < 4) {
#pragma unroll 1
            for (int c = 0; c < rows; c += 16) {
                float v[16];
                tmem_ld_32x32b_x16_wait(quarter + c, v);
                if (mine) finish<16>(a, m0 + c, n, min(16, rows - c), v, sw, bias);
            }
        }
    } else {
        // parts[m][n]: 128 fp32 numbers for each output row
        if (w < 4) {
            const uint32_t at = stages + 4 * (uint32_t)(w * 32 + lane);
#pragma unroll 1
            for (int c = 0; c < rows; c += 16) {
                float v[16];
                tmem_ld_32x32b_x16_wait(quarter + c, v);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + (c + j) * 512), "f"(v[j]) : "memory");
            }
        }
        __syncwarp();
        cluster_sync();
        if (w < 4) {
            const int c0 = rows * (int)rank / (int)S, c1 = rows * (int)(rank + 1) / (int)S;
#pragma unroll 1
            for (int c = c0; c < c1; c += 8) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.0f;
                for (uint32_t q = 0; q < S; ++q) {
                    const uint32_t at = map_to(stages + 4 * (uint32_t)(w * 32 + lane), q);
                    float p[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = c + j < c1 ? ld_cluster(at + (c + j) * 512) : 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += p[j];
                }
                if (mine) finish<8>(a, m0 + c, n, min(8, c1 - c), v, sw, bias);
            }
        }
        __syncwarp();
        cluster_sync();  // the others have read this block's parts
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 5) tmem_dealloc(tmem, T::kCols);
}

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
    return fn(m, t, 2, const_cast<void *>(p), dims, &pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN, bool CODES>
cudaError_t launch(const LinearArgs &a, const void *x, int64_t x_stride, const void *w,
                   int64_t w_stride, int sms, cudaStream_t s) {
    using T = Tile<TN>;
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(linear_kernel<TN, CODES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 T::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) set[dev] = true;
    }
    CUtensorMap wmap, xmap;
    if (!rows_map(&wmap, w, w_stride, a.N, a.K, a.type, kRowsW) ||
        !rows_map(&xmap, x, x_stride, a.M, a.K, a.type, TN))
        return cudaErrorNotSupported;
    const int tiles_n = (a.N + kRowsW - 1) / kRowsW, tiles_m = (a.M + TN - 1) / TN;
    const int kb = (a.K * (CODES ? 1 : 2) + kLine - 1) / kLine;
    // Blocks that share a tile: as many as fill the GPU about twice over (two blocks of a few
    // tokens lie on an SM), each with a few stages at least.
    int S = 1;
    while (S < 8 && (int64_t)tiles_n * tiles_m * S * 2 <= 2 * sms && kb >= 8 * S) S *= 2;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(tiles_n * S), (unsigned)tiles_m);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = T::kSmem;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)S;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.numAttrs = 1;
    c.attrs = &at;
    return cudaLaunchKernelEx(&c, linear_kernel<TN, CODES>, wmap, xmap, a);
}

template <bool CODES>
cudaError_t by_rows(const LinearArgs &a, const void *x, int64_t xs, const void *w, int64_t ws, int sms,
                    cudaStream_t s) {
    if (a.M <= 16) return launch<16, CODES>(a, x, xs, w, ws, sms, s);
    if (a.M <= 32) return launch<32, CODES>(a, x, xs, w, ws, sms, s);
    if (a.M <= 64) return launch<64, CODES>(a, x, xs, w, ws, sms, s);
    if (a.M <= 128) return launch<128, CODES>(a, x, xs, w, ws, sms, s);
    return launch<256, CODES>(a, x, xs, w, ws, sms, s);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, const void *x, int64_t x_stride, const void *w,
                          int64_t w_stride, int sms, cudaStream_t s) {
    return a.type == MOE_T_E4M3 ? by_rows<true>(a, x, x_stride, w, w_stride, sms, s)
                                : by_rows<false>(a, x, x_stride, w, w_stride, sms, s);
}

}  // namespace moe
