// Host side of include/moe_layer.h: argument checks and launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <cstdlib>

#include "layer.cuh"

using namespace moe;

namespace {

constexpr int kMostRows = 1 << 20;

bool number_type(int t) { return t == MOE_T_BF16 || t == MOE_T_F32 || t == MOE_T_F16; }
int size_of(int t) { return t == MOE_T_F32 ? 4 : t == MOE_T_E4M3 ? 1 : 2; }
bool at(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// A matrix of rows x cols: type and stride (which one row does not use).
bool matrix_ok(int type, int64_t stride, int rows, int cols) {
    return number_type(type) && (rows <= 1 || (stride >= cols && stride <= ((int64_t)1 << 40)));
}

int done(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
cudaStream_t str(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

int moe_add_norm(const void *x, int x_type, int64_t x_stride, const void *residual,
                 int residual_type, int64_t residual_stride, const void *weight, int weight_type,
                 float eps, int rows, int hidden, void *residual_out,
                 int64_t residual_out_stride, void *out, int out_type, int64_t out_stride,
                 uint8_t *codes, int64_t codes_stride, float *scales, moe_stream_t stream) {
    if (rows < 0 || rows > kMostRows || hidden < 1 || hidden > 32768) return MOE_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return MOE_ERR_SHAPE;
    if (!matrix_ok(x_type, x_stride, rows, hidden)) return MOE_ERR_SHAPE;
    if (residual && !matrix_ok(residual_type, residual_stride, rows, hidden)) return MOE_ERR_SHAPE;
    if (residual_out && (!residual || !matrix_ok(residual_type, residual_out_stride, rows, hidden)))
        return MOE_ERR_SHAPE;
    if (weight && !number_type(weight_type)) return MOE_ERR_SHAPE;
    if (out && !matrix_ok(out_type, out_stride, rows, hidden)) return MOE_ERR_SHAPE;
    if (codes && !matrix_ok(MOE_T_BF16, codes_stride, rows, hidden)) return MOE_ERR_SHAPE;
    if ((!codes) != (!scales)) return MOE_ERR_NULL;
    if (rows == 0) return MOE_OK;
    if (!x) return MOE_ERR_NULL;
    if (!residual_out && !out && !codes) return MOE_OK;
    if (!at(x, size_of(x_type)) || (residual && (!at(residual, size_of(residual_type)) ||
                                                 !at(residual_out, size_of(residual_type)))) ||
        (weight && !at(weight, size_of(weight_type))) || (out && !at(out, size_of(out_type))) ||
        !at(scales, 4))
        return MOE_ERR_ALIGN;
    int sms;
    const int rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    AddNormArgs a{};
    // (with one row a stride is not used)
    a.x = MatIn{x, x_stride, x_type};
    a.residual = MatIn{residual, residual_stride, residual_type};
    a.weight = weight;
    a.weight_type = weight_type;
    a.eps = eps;
    a.inv_hidden = (float)(1.0 / hidden);
    a.rows = rows;
    a.hidden = hidden;
    a.residual_out = MatOut{residual_out, residual_out_stride, residual_type};
    a.out = MatOut{out, out_stride, out_type};
    a.codes = codes;
    a.codes_stride = codes_stride;
    a.scales = scales;
    return done(launch_add_norm(a, sms, str(stream)));
}

int moe_linear(const void *x, int64_t x_stride, const float *x_scale, const void *w,
               int64_t w_stride, const float *w_scale, int type, const float *bias,
               int activation, const void *gate, int gate_type, int64_t gate_stride,
               const void *residual, int residual_type, int64_t residual_stride, void *out,
               int out_type, int64_t out_stride, int M, int N, int K, uint32_t *err,
               moe_stream_t stream) {
    if (M < 0 || M > kMostRows || N < 1 || N > kMostRows || K < 1 || K > kMostRows) return MOE_ERR_SHAPE;
    if (type != MOE_T_BF16 && type != MOE_T_F16 && type != MOE_T_E4M3) return MOE_ERR_SHAPE;
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_GELU) return MOE_ERR_SHAPE;
    // (tensor map strides end at 2^40 bytes)
    const int64_t most = ((int64_t)1 << 38);
    if ((M > 1 && (x_stride < K || x_stride > most)) || (N > 1 && (w_stride < K || w_stride > most)))
        return MOE_ERR_SHAPE;
    if (gate && !matrix_ok(gate_type, gate_stride, M, N)) return MOE_ERR_SHAPE;
    if (residual && !matrix_ok(residual_type, residual_stride, M, N)) return MOE_ERR_SHAPE;
    if (!matrix_ok(out_type, out_stride, M, N)) return MOE_ERR_SHAPE;
    if (M == 0) return MOE_OK;
    if (!x || !w || !out) return MOE_ERR_NULL;
    const int64_t pitch = 16 / size_of(type);
    if (!at(x, 16) || !at(w, 16) || (M > 1 && x_stride % pitch) || (N > 1 && w_stride % pitch) ||
        !at(x_scale, 4) || !at(w_scale, 4) || !at(bias, 4) || !at(out, size_of(out_type)) ||
        (gate && !at(gate, size_of(gate_type))) || (residual && !at(residual, size_of(residual_type))) ||
        !at(err, 4))
        return MOE_ERR_ALIGN;
    int sms;
    const int rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    LinearArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.type = type;
    a.activation = activation;
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.bias = bias;
    a.gate = MatIn{gate, gate_stride, gate_type};
    a.residual = MatIn{residual, residual_stride, residual_type};
    a.out = MatOut{out, out_stride, out_type};
    a.err = err;
    a.skip_line = -1;
#ifdef MOE_DEBUG_BOUNDS
    if (const char *v = getenv("MOE_LINEAR_DEBUG_SKIP_LINE")) a.skip_line = atoi(v);
#endif
    return done(launch_linear(a, x, x_stride, w, w_stride, sms, str(stream)));
}

int moe_linear_last_kernel(void) { return linear_last_kernel(); }

int moe_route_experts(const void *logits, int type, int64_t stride, const float *bias, int M,
                      int E, int top_k, int scoring, int groups, int top_groups, int group_best,
                      int renormalize, float scale, int32_t *topk_ids, float *topk_weights,
                      moe_stream_t stream) {
    if (M < 0 || M > kMostRows || E < 1 || E > 1024) return MOE_ERR_SHAPE;
    if (!matrix_ok(type, stride, M, E)) return MOE_ERR_SHAPE;
    if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID) return MOE_ERR_SHAPE;
    if (groups < 1 || groups > 32 || E % groups || top_groups < 1 || top_groups > groups ||
        (group_best != 1 && group_best != 2) || (renormalize != 0 && renormalize != 1))
        return MOE_ERR_SHAPE;
    if (top_k < 1 || top_k > 32 || top_k > E / groups * top_groups) return MOE_ERR_SHAPE;
    if (!std::isfinite(scale)) return MOE_ERR_SHAPE;
    if (M == 0) return MOE_OK;
    if (!logits || !topk_ids || !topk_weights) return MOE_ERR_NULL;
    if (!at(logits, size_of(type)) || !at(bias, 4) || !at(topk_ids, 4) || !at(topk_weights, 4))
        return MOE_ERR_ALIGN;
    int sms;
    const int rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    RouteExpertsArgs a{};
    a.logits = logits;
    a.type = type;
    a.stride = stride;
    a.bias = bias;
    a.M = M;
    a.E = E;
    a.top_k = top_k;
    a.scoring = scoring;
    a.groups = groups;
    a.top_groups = top_groups;
    a.group_best = group_best;
    a.renormalize = renormalize;
    a.scale = scale;
    a.ids = topk_ids;
    a.weights = topk_weights;
    return done(launch_route_experts(a, sms, str(stream)));
}

}  // extern "C"
