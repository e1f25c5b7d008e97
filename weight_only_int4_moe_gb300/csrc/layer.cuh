// Arguments and launchers of the operators of include/moe_layer.h, and element access
// by type, between layer_abi.cu and the kernels' files.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device.cuh"
#include "kernels.cuh"
#include "moe_layer.h"

namespace moe {

// A matrix of rows of contiguous elements; p NULL: absent.
struct MatIn {
    const void *p;
    int64_t stride;
    int type;
};
struct MatOut {
    void *p;
    int64_t stride;
    int type;
};

MOE_DEV float load_as_float(const void *p, int type, int64_t i) {
    if (type == MOE_T_F32) return reinterpret_cast<const float *>(p)[i];
    const uint16_t v = reinterpret_cast<const uint16_t *>(p)[i];
    return type == MOE_T_BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}
MOE_DEV uint16_t to_bits16(float v, int type) {
    return type == MOE_T_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                              : __half_as_ushort(__float2half_rn(v));
}

struct AddNormArgs {
    MatIn x, residual;
    const void *weight;
    int weight_type;
    float eps, inv_hidden;
    int rows, hidden;
    MatOut residual_out, out;
    uint8_t *codes;
    int64_t codes_stride;
    float *scales;
    int stride8;  // of the rows, modulo 8 (ENDS kernels)
};

struct LinearArgs {
    int M, N, K, type, activation;
    const float *x_scale, *w_scale, *bias;
    MatIn gate, residual;
    MatOut out;
    uint32_t *err;
    bool vec_gate, vec_residual, vec_out;  // four neighbours of a row may be one access
    bool vec2;  // two may, in each of the three
    // Debug-bounds builds: block 0 leaves the copy of w for its i-th line out, so that a wait runs
    // out.  -1: none.
    int skip_line;
};

struct RouteExpertsArgs {
    const void *logits;
    int type;
    int64_t stride;
    const float *bias;
    int M, E, top_k, scoring, groups, top_groups, group_best, renormalize;
    float scale;
    int32_t *ids;
    float *weights;
};

// How an add and norm's rows lie: vectors of eight throughout, vectors but for the ends, or
// neither.
enum class Grid { kVectors, kEnds, kNone };
template <int TX>
cudaError_t add_norm_of(const AddNormArgs &a, Grid grid, int sms, cudaStream_t s);
cudaError_t launch_add_norm(AddNormArgs a, int sms, cudaStream_t s);
// cudaErrorNotSupported: the operands' tensor maps could not be made.
cudaError_t launch_linear(LinearArgs a, const void *x, int64_t x_stride, const void *w,
                          int64_t w_stride, int sms, cudaStream_t s);
int linear_last_kernel();
cudaError_t launch_route_experts(const RouteExpertsArgs &a, int sms, cudaStream_t s);

}  // namespace moe
