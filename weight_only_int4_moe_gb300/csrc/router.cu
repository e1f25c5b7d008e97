// Routing to experts (moe_route_experts): scores, a bias for balance, groups, top-k,
// renormalised weights.
//
// A warp has a token; lane l holds experts l, l + 32, ...  The kernel reads M E logits and
// writes 8 M top_k bytes; what costs is choosing.  The lanes' largest keys are sorted across
// the warp: the top_k experts lie at or above the top_k-th of them, and seldom more than half
// as many again do.  These candidates move to a lane each (in index order) and count who is
// before them.
//
// Which experts are chosen must not depend on how an exponential was rounded.  Without a bias
// the scores order as the logits do, and the logits are the keys.  With one, c = s + bias is
// formed in fp32, whose error against the real number is bounded (`unsure`, and c's own
// rounding); where two neighbours in the order are nearer to each other than that, the
// candidates are compared again in 64 bits.  That is seldom: the 9 gaps of a top-8 choice are
// some 1e-2 wide.  A group's sum of two c is off by the roundings of its terms, which may be far
// larger than the sum (biases of either sign).  So each group has a bound of its own, and the
// groups whose intervals reach the border between chosen and other ones are compared in 64 bits.
//
// Measured: 8192 tokens of 384 experts, sigmoid and bias, 14 us, of them 2 for the dozen near
// ties (each 1 to 2 us of 64-bit latency in one warp); 1130 instructions a token, 58 % of the issue
// slots.  One token 3.1 us.  4096 tokens, 4 of 8 groups of 32: 12.3 us.  bf16 logits with equal
// biases, where most tokens have ties, 25 us.
#include <cfloat>

#include "layer.cuh"

namespace moe {

namespace {

constexpr int kWarps = 2;
constexpr uint32_t kGone = 0;              // the key of what is taken or not open
constexpr uint32_t kMasked = 0x007FFFFFu;  // of -inf: what is not available

// A key that orders as the float does (no NaN; -0 is below +0).
MOE_DEV uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
MOE_DEV float value_of(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

// A logit: NaN counts as -inf (not available), +inf as the largest number.
MOE_DEV float logit_of(const RouteExpertsArgs &a, int64_t row, int e) {
    const float x = load_as_float(a.logits, a.type, row * a.stride + e);
    return isnan(x) ? -INFINITY : fminf(x, FLT_MAX);
}
MOE_DEV float sigmoid(float x) {
    const float t = expf(-fabsf(x));
    return (x < 0.0f ? t : 1.0f) / (1.0f + t);
}
MOE_DEV double sigmoid(double x) {
    const double t = exp(-fabs(x));
    return (x < 0.0 ? t : 1.0) / (1.0 + t);
}
// With the hardware's exponential (2^-22 relative, and its argument's rounding, |x| 2^-23) and
// reciprocal (one step): s (1 - s) (2^-22 + |x| 2^-23) + 3 2^-24, within 3e-7.  Far below 0 the
// exponential is infinite and the score 0.
MOE_DEV float sigmoid_fast(float x) {
    float t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
    return r;
}
MOE_DEV float exp_fast(float x) {
    float t;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(x * 1.4426950408889634f));
    return t;
}

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

// The softmax's top and 1 / sum in 64 bits (0 and 1 for the sigmoid).
MOE_DEV void softmax_exactly(const RouteExpertsArgs &a, int64_t row, int lane, double &top, double &inv) {
    top = 0.0;
    inv = 1.0;
    if (a.scoring != MOE_SCORE_SOFTMAX) return;
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, logit_of(a, row, e));
    m = warp_max(m);
    top = m == -INFINITY ? 0.0 : (double)m;
    double sum = 0.0;
#pragma unroll 4
    for (int e = lane; e < a.E; e += 32) sum += exp((double)logit_of(a, row, e) - top);
    sum = warp_sum(sum);
    inv = sum > 0.0 ? 1.0 / sum : 0.0;
}
// An expert's c in 64 bits, -inf where it is not available.
MOE_DEV double score_exactly(const RouteExpertsArgs &a, int64_t row, int e, double top, double inv) {
    const float l = logit_of(a, row, e), b = a.bias ? a.bias[e] : 0.0f;
    const double s = a.scoring == MOE_SCORE_SOFTMAX ? exp((double)l - top) * inv : sigmoid((double)l);
    return l > -INFINITY && b > -INFINITY ? s + (double)b : -INFINITY;
}

// The candidates of a token in 64 bits: lane j < n has expert e (ascending in j).  -> the
// lane's expert in the order of choice; list: room for 32.
__device__ __noinline__ int order_exactly(const RouteExpertsArgs &a, int64_t row, int lane, int n, int e,
                                          int *list) {
    double top, inv;
    softmax_exactly(a, row, lane, top, inv);
    const double c = lane < n ? score_exactly(a, row, e, top, inv) : -INFINITY;
    int before = 0;
    for (int j = 0; j < n; ++j) {
        const double o = __shfl_sync(0xffffffffu, c, j);
        before += o > c || (o == c && j < lane);
    }
    __syncwarp();
    if (lane < n) list[before] = e;
    __syncwarp();
    return list[lane];
}

// The groups of a token where fp32 leaves some open: `surely` are chosen, and of those in `close`
// the best, by their best experts' c in 64 bits: lane j < n has one, expert e.  -> the chosen
// groups.
__device__ __noinline__ uint32_t groups_exactly(const RouteExpertsArgs &a, int64_t row, int lane, int n,
                                                int e, uint32_t surely, uint32_t close) {
    double top, inv;
    softmax_exactly(a, row, lane, top, inv);
    const double c = lane < n ? score_exactly(a, row, e, top, inv) : -INFINITY;
    const int mine = lane < n ? e / (a.E / a.groups) : -1;
    double of_group = -INFINITY;
    for (uint32_t left = close; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        double x = mine == g ? c : -INFINITY, y = -INFINITY;  // the two best
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double x2 = __shfl_xor_sync(0xffffffffu, x, o);
            const double y2 = __shfl_xor_sync(0xffffffffu, y, o);
            y = fmax(fmin(x, x2), fmax(y, y2));
            x = fmax(x, x2);
        }
        if (lane == g) of_group = a.group_best == 2 && y > -INFINITY ? x + y : x;
    }
    int before = __popc(surely);
    for (uint32_t left = close; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        const double o = __shfl_sync(0xffffffffu, of_group, g);
        before += o > of_group || (o == of_group && g < lane);
    }
    return surely | __ballot_sync(0xffffffffu, ((close >> lane) & 1u) && before < a.top_groups);
}

// The whole choice in 64 bits; c: room for E numbers.  -> the lane's expert.
__device__ __noinline__ int choose_exactly(const RouteExpertsArgs &a, int64_t row, int lane, double *c) {
    double top, inv;
    softmax_exactly(a, row, lane, top, inv);
#pragma unroll 4
    for (int e = lane; e < a.E; e += 32) c[e] = score_exactly(a, row, e, top, inv);
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

// Descending order of a value a lane across the warp.
MOE_DEV uint32_t sort_lanes(uint32_t v, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int j = k / 2; j; j /= 2) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
            const bool larger = ((lane & j) == 0) == ((lane & k) == 0);
            v = larger ? max(v, o) : min(v, o);
        }
    return v;
}

// What the keys are made of.
constexpr int kLogits = 0, kSigmoid = 1, kSoftmax = 2;

// V: experts of a lane.
template <int V, int KEYS>
__global__ void __launch_bounds__(32 * kWarps, V <= 12 ? 14 : V <= 16 ? 8 : 4)
    route_experts_kernel(const RouteExpertsArgs a) {
    extern __shared__ uint2 room[];  // of a warp: E pairs (key, expert), or E 64-bit numbers
    __shared__ int order[kWarps][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint2 *const list = room + (size_t)w * a.E;
    const uint32_t below = (1u << lane) - 1u;
    const int size = a.E / a.groups;
    const float per_group = 1.0f / (float)size;
    const bool soft = KEYS == kSoftmax || (KEYS == kLogits && a.scoring == MOE_SCORE_SOFTMAX);
    const bool sums = KEYS != kLogits && a.groups > 1 && a.group_best == 2 && size > 1;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + w; t < a.M; t += (int64_t)gridDim.x * kWarps) {
        float l[V], b[V];
        uint32_t key[V];
        if (a.type == MOE_T_F32) {
            const float *p = reinterpret_cast<const float *>(a.logits) + t * a.stride + lane;
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < a.E ? p[32 * i] : -INFINITY;
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(a.logits) + t * a.stride + lane;
            uint16_t r[V];
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = lane + 32 * i < a.E ? p[32 * i] : (uint16_t)0xFFFFu;
            // (all ones are NaN in either type)
            if (a.type == MOE_T_BF16) {
#pragma unroll
                for (int i = 0; i < V; ++i) l[i] = __uint_as_float((uint32_t)r[i] << 16);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) l[i] = __half2float(__ushort_as_half(r[i]));
            }
        }
        if (KEYS != kLogits) {
#pragma unroll
            for (int i = 0; i < V; ++i) b[i] = a.bias && lane + 32 * i < a.E ? a.bias[lane + 32 * i] : 0.0f;
        }
        if (KEYS != kSigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = l[i] > -INFINITY ? fminf(l[i], FLT_MAX) : -INFINITY;
        }
        float top = 0.0f, inv = 1.0f;
        if (KEYS == kSoftmax || (soft && !a.renormalize)) {
            top = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
            top = warp_max(top);
            if (top == -INFINITY) top = 0.0f;
            // (of the approximate exponentials: the weights divided by it are within 3e-6, of which
            // the 37 additions are most; renormalised ones do not use it)
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += exp_fast(l[i] - top);
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        }
        // bounds the error of the difference of two scores (the softmax's by its largest, and
        // by the sum's 37 additions at most); c adds its own rounding
        const float unsure = KEYS == kSoftmax ? 4e-6f * inv : 1e-6f;
        bool sure = true;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float c = l[i] + 0.0f;  // (-0 and +0 are equal)
            if (KEYS == kSigmoid) c = sigmoid_fast(l[i]) + b[i];
            if (KEYS == kSoftmax) c = exp_fast(l[i] - top) * inv + b[i];
            if (KEYS != kLogits) c = l[i] > -INFINITY && c > -INFINITY ? c : -INFINITY;
            key[i] = lane + 32 * i < a.E ? key_of(c) : kGone;
        }
        if (a.groups > 1) {
            float mine = -INFINITY, slack = 0.0f;  // lane g: group g's value, and a bound on its error
            uint32_t least = kMasked;  // the last of the group's experts that count
            // the warp's two best of a group -> its value, in lane g
            auto value = [&](int g, uint32_t x, uint32_t y) {
                const uint32_t best = __reduce_max_sync(0xffffffffu, x);
                uint32_t second = 0;
                if (sums) {
                    const uint32_t who = __ballot_sync(0xffffffffu, x == best);
                    second = __popc(who) > 1 ? best : __reduce_max_sync(0xffffffffu, x == best ? y : x);
                }
                if (lane == g) least = sums ? second : best;
                if (lane == g && best > kMasked) {
                    const float b = value_of(best), s = second > kMasked ? value_of(second) : 0.0f;
                    // (a sum of numbers beyond fp32 is unsure, not infinite)
                    mine = b < INFINITY ? fminf(fmaxf(b + s, -FLT_MAX), FLT_MAX) : b;
                    // two scores; the roundings of the two c, of their sum and of the interval's ends
                    // below, each 2^-24 of the terms at most
                    slack = b < INFINITY ? unsure + 2e-7f * (fabsf(b) + fabsf(s)) : 0.0f;
                }
            };
            if (size % 32 == 0) {
                // a group is some of every lane's registers
                uint32_t x = 0, y = 0;
                int g = 0, left = size / 32;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    y = max(y, min(x, key[i]));
                    x = max(x, key[i]);
                    if (--left == 0 && g < a.groups) {
                        value(g++, x, y);
                        x = y = 0;
                        left = size / 32;
                    }
                }
            } else {
                for (int g = 0; g < a.groups; ++g) {
                    uint32_t x = 0, y = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const uint32_t k = (uint32_t)(lane + 32 * i - g * size) < (uint32_t)size ? key[i] : 0u;
                        y = max(y, min(x, k));
                        x = max(x, k);
                    }
                    value(g, x, y);
                }
            }
            float gap, edge;
            uint32_t open = choose_groups(a, mine, lane, gap, edge);
            if (KEYS != kLogits) {
                // (-inf: fewer groups than that have an expert left)
                const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(slack)));
                uint32_t surely = 0, close = 0;
                if (!(gap > 2.0f * most) && edge > -INFINITY) {
                    // which groups surely are among the best, and which surely are not
                    const bool finite = fabsf(mine) < INFINITY;
                    const float lo = finite ? fmaxf(mine - slack, -FLT_MAX) : mine;
                    const float hi = finite ? fminf(mine + slack, FLT_MAX) : mine;
                    int may = 0, must = 0;  // groups that may, and that must, be before this one
                    for (int g = 0; g < a.groups; ++g) {
                        const float h = __shfl_sync(0xffffffffu, hi, g), l = __shfl_sync(0xffffffffu, lo, g);
                        may += h >= lo ? 1 : 0;  // (itself among them)
                        must += l > hi ? 1 : 0;
                    }
                    surely = __ballot_sync(0xffffffffu, lane < a.groups && may <= a.top_groups);
                    close = __ballot_sync(0xffffffffu,
                                          lane < a.groups && may > a.top_groups && must < a.top_groups);
                }
                if (close) {
                    if (least > kMasked) {
                        const float v = value_of(least);
                        if (v < INFINITY) least = key_of(v - (unsure + 2.5e-7f * fabsf(v)));
                    }
                    least = max(least, kMasked + 1u);
                    int m = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int g = (int)(((float)(lane + 32 * i) + 0.5f) * per_group) & 31;
                        const bool in = key[i] >= __shfl_sync(0xffffffffu, least, g) && ((close >> g) & 1u);
                        const uint32_t who = __ballot_sync(0xffffffffu, in);
                        if (in) list[m + __popc(who & below)] = make_uint2(0u, (uint32_t)(lane + 32 * i));
                        m += __popc(who);
                    }
                    __syncwarp();
                    if (m <= 32)
                        open = groups_exactly(a, t, lane, m, lane < m ? (int)list[lane].y : 0, surely, close);
                    else
                        sure = false;
                    __syncwarp();
                }
            }
            if (KEYS != kLogits && !a.bias) {
                // inside the groups the logits decide
#pragma unroll
                for (int i = 0; i < V; ++i)
                    key[i] = lane + 32 * i < a.E ? key_of(logit_of(a, t, lane + 32 * i) + 0.0f) : kGone;
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                // e / size: E is at most 1024, so the product is off by less than 1 / (2 size)
                if (!((open >> (int)(((float)(lane + 32 * i) + 0.5f) * per_group)) & 1u)) key[i] = kGone;
        }

        // the next expert behind the chosen ones counts too, where keys are scores
        const bool scored = KEYS != kLogits && a.bias;
        const int want = scored ? a.top_k + 1 : a.top_k;
        uint32_t floor_key = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) floor_key = max(floor_key, key[i]);
        floor_key = want <= 32 ? __shfl_sync(0xffffffffu, sort_lanes(floor_key, lane), want - 1) : 0u;
        floor_key = max(floor_key, kMasked);
        int chosen = 0, n = 0;
        // lists the keys that are no smaller than floor_key, in index order -> how many
        auto gather = [&]() {
            int m = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool in = key[i] >= floor_key;
                const uint32_t who = __ballot_sync(0xffffffffu, in);
                if (in) list[m + __popc(who & below)] = make_uint2(key[i], (uint32_t)(lane + 32 * i));
                m += __popc(who);
            }
            __syncwarp();
            return m;
        };
        if (sure) {
            n = gather();
            if (n <= 32) {
                const uint2 own = lane < n ? list[lane] : make_uint2(kGone, 0u);
                int before = 0;
                for (int j = 0; j < n; ++j)  // (keys end below the largest number)
                    before += __shfl_sync(0xffffffffu, own.x, j) + (j < lane) > own.x;
                __syncwarp();
                if (lane < n) list[before] = own;
                __syncwarp();
                const uint2 sorted = lane < n ? list[lane] : make_uint2(kGone, 0u);
                chosen = (int)sorted.y;
                if (scored) {
                    const float c = value_of(sorted.x), prev = __shfl_up_sync(0xffffffffu, c, 1);
                    const bool close = lane > 0 && lane < want && lane < n && sorted.x > kMasked &&
                                       !(prev - c > unsure + 2.5e-7f * fabsf(prev));
                    if (__any_sync(0xffffffffu, close)) {
                        // all that may belong to the chosen ones: whatever is not surely less
                        // than the last of them
                        const float last = __shfl_sync(0xffffffffu, c, a.top_k - 1);
                        if (last > -INFINITY)  // (NaN: fewer than top_k are available)
                            floor_key = min(floor_key, key_of(last - (unsure + 2.5e-7f * fabsf(last))));
                        __syncwarp();
                        n = gather();
                        if (n <= 32)
                            chosen = order_exactly(a, t, lane, n, lane < n ? (int)list[lane].y : 0, order[w]);
                    }
                }
            }
            // many equal ones, or more than 31 of them wanted
            if (n > 32 && scored) sure = false;
        }
        if (!sure) {
            chosen = choose_exactly(a, t, lane, reinterpret_cast<double *>(list));
        } else if (n > 32) {
            uint32_t best = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = lane + 32 * i;
                }
            for (int j = 0; j < a.top_k; ++j) {
                const uint32_t k = __reduce_max_sync(0xffffffffu, best);
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
        }

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
        __syncwarp();
    }
}

template <int V, int KEYS>
cudaError_t launch(const RouteExpertsArgs &a, int sms, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.M + kWarps - 1) / kWarps, most = (int64_t)sms * 32;
    auto c = pdl_config((unsigned)(blocks < most ? blocks : most), 32 * kWarps, (size_t)kWarps * a.E * 8, s);
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return cudaLaunchKernelEx(&c, route_experts_kernel<V, KEYS>, a);
}

template <int V>
cudaError_t by_keys(const RouteExpertsArgs &a, int sms, cudaStream_t s) {
    const bool sums = a.groups > 1 && a.group_best == 2 && a.groups < a.E;
    if (!a.bias && !sums) return launch<V, kLogits>(a, sms, s);
    return a.scoring == MOE_SCORE_SOFTMAX ? launch<V, kSoftmax>(a, sms, s) : launch<V, kSigmoid>(a, sms, s);
}

}  // namespace

cudaError_t launch_route_experts(const RouteExpertsArgs &a, int sms, cudaStream_t s) {
    if (a.E <= 64) return by_keys<2>(a, sms, s);
    if (a.E <= 128) return by_keys<4>(a, sms, s);
    if (a.E <= 256) return by_keys<8>(a, sms, s);
    if (a.E <= 384) return by_keys<12>(a, sms, s);
    if (a.E <= 512) return by_keys<16>(a, sms, s);
    return by_keys<32>(a, sms, s);
}

}  // namespace moe
