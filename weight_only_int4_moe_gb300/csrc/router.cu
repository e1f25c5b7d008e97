// Routing to experts (moe_route_experts): scores, a bias for balance, groups, top-k,
// renormalised weights.
//
// A warp has a token; lane l holds experts l, l + 32, ...  The kernel reads M E logits and
// writes 8 M top_k bytes; what costs is choosing: each of the top_k rounds takes the warp's
// largest remaining key and, among equal ones, the lowest index (two warp reductions).
//
// Which experts are chosen must not depend on how an exponential was rounded.  Without a bias
// the scores order as the logits do, and the logits are the keys.  With one, c = s + bias is
// formed in fp32, whose error against the real number is bounded (`unsure`); where two
// neighbours in the order are nearer to each other than that, the token is done again in 64
// bits.  That is seldom: the 9 gaps of a top-8 choice are some 1e-2 wide.
#include <cfloat>

#include "layer.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;
constexpr uint32_t kGone = 0, kMasked = 1;  // keys of what is taken or not open, and not available

// A key that orders as the float does (numbers only), above kMasked.
MOE_DEV uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // (-0 and +0 are equal)
    return (u >> 31) ? ~u : u | 0x80000000u;
}
MOE_DEV float value_of(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

// A logit: NaN counts as -inf (not available), +inf as the largest number.
MOE_DEV float logit_of(const RouteExpertsArgs &a, int64_t row, int e) {
    const float x = load_as_float(a.logits, a.type, row * a.stride + e);
    return isnan(x) ? -INFINITY : fminf(x, FLT_MAX);
}
MOE_DEV float sigmoid(float x) { return expf(fminf(x, 0.0f)) / (1.0f + expf(-fabsf(x))); }
MOE_DEV double sigmoid(double x) { return exp(fmin(x, 0.0)) / (1.0 + exp(-fabs(x))); }

MOE_DEV float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <typename F>
MOE_DEV F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Which groups are chosen, as bits: lane g holds group g's value.  -> the gap between the
// last chosen and the first other one.
template <typename F>
MOE_DEV uint32_t choose_groups(const RouteExpertsArgs &a, F value, int lane, F &gap, F &edge) {
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
        const F o = __shfl_sync(0xffffffffu, value, g);
        before += o > value || (o == value && g < lane);
    }
    const bool in = lane < a.groups;
    const uint32_t last = __ballot_sync(0xffffffffu, in && before == a.top_groups - 1);
    const uint32_t next = __ballot_sync(0xffffffffu, in && before == a.top_groups);
    edge = __shfl_sync(0xffffffffu, value, __ffs(last) - 1);
    gap = next ? edge - __shfl_sync(0xffffffffu, value, next ? __ffs(next) - 1 : 0) : (F)INFINITY;
    return __ballot_sync(0xffffffffu, in && before < a.top_groups);
}

// The whole choice in 64 bits; c: room for E numbers.  -> the lane's expert.
__device__ __noinline__ int choose_exactly(const RouteExpertsArgs &a, int64_t row, int lane, double *c) {
    double top = -INFINITY, inv = 0.0;
    if (a.scoring == MOE_SCORE_SOFTMAX) {
        float m = -INFINITY;
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, logit_of(a, row, e));
        m = warp_max(m);
        top = m == -INFINITY ? 0.0 : (double)m;
        double sum = 0.0;
        for (int e = lane; e < a.E; e += 32) sum += exp((double)logit_of(a, row, e) - top);
        sum = warp_sum(sum);
        inv = sum > 0.0 ? 1.0 / sum : 0.0;
    }
    for (int e = lane; e < a.E; e += 32) {
        const float l = logit_of(a, row, e), b = a.bias ? a.bias[e] : 0.0f;
        const double s = a.scoring == MOE_SCORE_SOFTMAX ? exp((double)l - top) * inv : sigmoid((double)l);
        const bool here = l > -INFINITY && b > -INFINITY;
        c[e] = here ? s + (double)b : -INFINITY;
    }
    __syncwarp();
    uint32_t open = 0xffffffffu;
    const int size = a.E / a.groups;
    if (a.groups > 1) {
        double mine = -INFINITY;
        for (int g = 0; g < a.groups; ++g) {
            double x = -INFINITY, y = -INFINITY;  // the two best
            for (int e = g * size + lane; e < (g + 1) * size; e += 32) {
                const double v = c[e];
                y = fmax(y, fmin(x, v));
                x = fmax(x, v);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const double x2 = __shfl_xor_sync(0xffffffffu, x, o);
                const double y2 = __shfl_xor_sync(0xffffffffu, y, o);
                y = fmax(fmin(x, x2), fmax(y, y2));
                x = fmax(x, x2);
            }
            if (lane == g) mine = a.group_best == 2 && y > -INFINITY ? x + y : x;
        }
        double gap, edge;
        open = choose_groups(a, mine, lane, gap, edge);
    }
    __syncwarp();
    // the keys: NaN for what is taken or not open
    for (int e = lane; e < a.E; e += 32) {
        if (!a.bias) {
            const float l = logit_of(a, row, e);
            c[e] = (double)l;
        }
        if (!((open >> (e / size)) & 1u) && a.groups > 1) c[e] = NAN;
    }
    __syncwarp();
    int chosen = 0;
    for (int j = 0; j < a.top_k; ++j) {
        double best = -INFINITY;
        int at = 0x7fffffff;
        for (int e = lane; e < a.E; e += 32) {
            const double v = c[e];
            if (v == v && (at == 0x7fffffff || v > best)) {
                best = v;
                at = e;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double v = __shfl_xor_sync(0xffffffffu, best, o);
            const int i = __shfl_xor_sync(0xffffffffu, at, o);
            if (i != 0x7fffffff && (at == 0x7fffffff || v > best || (v == best && i < at))) {
                best = v;
                at = i;
            }
        }
        if (lane == j) chosen = at;
        if ((at & 31) == lane) c[at] = NAN;
        __syncwarp();
    }
    return chosen;
}

// V: experts of a lane.
template <int V>
__global__ void __launch_bounds__(32 * kWarps) route_experts_kernel(const RouteExpertsArgs a) {
    extern __shared__ double exact[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int size = a.E / a.groups;
    const bool soft = a.scoring == MOE_SCORE_SOFTMAX;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + w; t < a.M; t += (int64_t)gridDim.x * kWarps) {
        float l[V];
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < a.E ? logit_of(a, t, e) : -INFINITY;
        }
        float top = 0.0f, inv = 1.0f;
        if (soft) {
            top = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
            top = warp_max(top);
            if (top == -INFINITY) top = 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += expf(l[i] - top);
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        }
        // the largest score bounds every score's error; c adds its own rounding
        const float unsure = soft ? 4e-6f * inv : 1e-6f;
        bool sure = true;
        uint32_t open = 0xffffffffu;
        const bool sums = a.groups > 1 && a.group_best == 2 && size > 1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            key[i] = kGone;
            if (e < a.E) {
                const float b = a.bias ? a.bias[e] : 0.0f;
                const bool here = l[i] > -INFINITY && b > -INFINITY;
                float c = l[i];
                if (a.bias || sums) c = (soft ? expf(l[i] - top) * inv : sigmoid(l[i])) + b;
                key[i] = here ? key_of(c) : kMasked;
            }
        }
        if (a.groups > 1) {
            float mine = -INFINITY;
            for (int g = 0; g < a.groups; ++g) {
                uint32_t x = 0, y = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane + 32 * i;
                    const uint32_t k = e >= g * size && e < (g + 1) * size ? key[i] : 0u;
                    y = max(y, min(x, k));
                    x = max(x, k);
                }
                const uint32_t best = __reduce_max_sync(0xffffffffu, x);
                const uint32_t who = __ballot_sync(0xffffffffu, x == best);
                uint32_t second = 0;
                if (sums)
                    second = __popc(who) > 1 ? best : __reduce_max_sync(0xffffffffu, x == best ? y : x);
                if (lane == g && best > kMasked)
                    mine = second > kMasked ? value_of(best) + value_of(second) : value_of(best);
            }
            float gap, edge;
            open = choose_groups(a, mine, lane, gap, edge);
            if ((a.bias || sums) && !(gap > 2.0f * unsure + 2.5e-7f * fabsf(edge))) sure = edge == -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                if (e < a.E) {
                    if (!a.bias && sums) key[i] = l[i] > -INFINITY ? key_of(l[i]) : kMasked;
                    if (!((open >> (e / size)) & 1u)) key[i] = kGone;
                }
            }
        }
        // top_k rounds, and one more to see how far the next expert is
        uint32_t best = 0;
        int at = 0;
        int chosen = 0;
        float last = 0.0f;
        const int rounds = a.bias ? a.top_k + 1 : a.top_k;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        for (int j = 0; j < rounds; ++j) {
            const uint32_t k = __reduce_max_sync(0xffffffffu, best);
            if (j < a.top_k) {
                const int e = (int)__reduce_min_sync(0xffffffffu, best == k ? (uint32_t)at : 0xffffffffu);
                if (lane == j) chosen = e;
                if (best == k && at == e) {
                    best = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (lane + 32 * i == e) key[i] = kGone;
                        if (key[i] > best) {
                            best = key[i];
                            at = lane + 32 * i;
                        }
                    }
                }
            }
            if (a.bias && k > kMasked) {
                const float c = value_of(k);
                if (j > 0 && !(last - c > unsure + 2.5e-7f * fabsf(last))) sure = false;
                last = c;
            }
        }
        if (!sure) chosen = choose_exactly(a, t, lane, exact + (size_t)w * a.E);

        const bool has = lane < a.top_k;
        const float x = has ? logit_of(a, t, chosen) : -INFINITY;
        const bool here = x > -INFINITY && !(a.bias && !(a.bias[has ? chosen : 0] > -INFINITY));
        float v;
        if (!a.renormalize) {
            v = soft ? expf(x - top) * inv : sigmoid(x);
        } else if (soft) {
            // the softmax over the chosen ones
            const float m = warp_max(here ? x : -INFINITY);
            v = expf(x - m);
        } else {
            // relative to e^min(x, 0) of the largest one
            const float y = fminf(x, 0.0f), m = warp_max(here ? y : -INFINITY);
            v = expf(y - m) / (1.0f + expf(-fabsf(x)));
        }
        v = here ? v : 0.0f;
        if (a.renormalize) {
            const float sum = warp_sum(v);
            v = sum > 0.0f ? v / sum : 0.0f;
        }
        if (has) {
            a.ids[t * a.top_k + lane] = chosen;
            a.weights[t * a.top_k + lane] = v * a.scale;
        }
    }
}

template <int V>
cudaError_t launch(const RouteExpertsArgs &a, int sms, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.M + kWarps - 1) / kWarps, most = (int64_t)sms * 16;
    route_experts_kernel<V><<<(unsigned)(blocks < most ? blocks : most), 32 * kWarps,
                              (size_t)kWarps * a.E * 8, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_experts(const RouteExpertsArgs &a, int sms, cudaStream_t s) {
    if (a.E <= 64) return launch<2>(a, sms, s);
    if (a.E <= 128) return launch<4>(a, sms, s);
    if (a.E <= 256) return launch<8>(a, sms, s);
    if (a.E <= 384) return launch<12>(a, sms, s);
    if (a.E <= 512) return launch<16>(a, sms, s);
    return launch<32>(a, sms, s);
}

}  // namespace moe
