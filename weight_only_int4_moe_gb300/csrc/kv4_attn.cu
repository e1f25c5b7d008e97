// Attention over the 4-bit cache (include/moe_kv4.h): one warp per query row,
// 32 tokens at a time with a running maximum and sum.
#include "kv4_launch.cuh"

namespace moe {

namespace {

template <int D>
__global__ void __launch_bounds__(128) kv4_attn_kernel(const KvAttnArgs a) {
    constexpr int NG = D / 32, W = D / 8;  // words of a row
    __shared__ float sq[4][D];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int row = blockIdx.x * 4 + w;
    if (row >= a.batch.tokens * a.q_heads) return;
    const int t = row / a.q_heads, hq = row - t * a.q_heads, h = hq / a.group;
    const int b = kv_request_of(a.batch.cu_q, a.batch.requests, t);
    const int kv = min(a.batch.kv_len[b], (int)min((long long)a.batch.stride * a.pool.ps, 1ll << 30));
    const int len = a.batch.kv_len[b], first = len - (a.batch.cu_q[b + 1] - a.batch.cu_q[b]);
    const int p = first + t - a.batch.cu_q[b];
    const uint64_t tree = a.tree ? a.tree[t] : ~0ull;
    if (kv < len && lane == 0) kv_report(a.err, MOE_KV4_DEVERR_PAGE);  // beyond its table
    bool bad = false;
    for (int d = lane; d < D; d += 32) {
        float x = __uint_as_float((uint32_t)a.q[(size_t)t * a.q_stride + hq * D + d] << 16);
        bad |= !(fabsf(x) <= 65504.0f);
        sq[w][d] = fminf(fmaxf(x, -65504.0f), 65504.0f);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) kv_report(a.err, MOE_KV4_DEVERR_RANGE);
    __syncwarp();
    const int end = min(kv, p + 1);
    int j0 = a.window > 0 ? max(0, p - a.window + 1) : 0;
    j0 &= ~31;
    const int ps = a.pool.ps;
    float m = -INFINITY, sum = 0.0f, acc[4] = {};
    for (; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        bool see = j < end && (a.window <= 0 || j > p - a.window);
        if (a.tree && j >= first) see = see && (j - first < 64) && ((tree >> (j - first)) & 1);
        const int page = see ? kv_page_of(a.batch, a.pool, b, j, a.err) : -1;
        see = page >= 0;
        float x = -INFINITY;
        const uint8_t *blk = see ? kv_block(a.pool, page, h) : nullptr;
        const int slot = j % ps;
        if (see) {
            const uint32_t *kr = reinterpret_cast<const uint32_t *>(blk + slot * (D / 2));
            const __half *sc = reinterpret_cast<const __half *>(blk + ps * D) + slot * NG;
            float dot = 0.0f;
            for (int g = 0; g < NG; ++g) {
                float part = 0.0f;
                for (int u = 0; u < 4; ++u) {
                    const uint32_t c = kr[u * NG + g];
                    const float *q = &sq[w][32 * g + 8 * u];
                    for (int i = 0; i < 4; ++i) {
                        part += q[2 * i] * (float)((int)((c >> (4 * i)) & 15) - 8);
                        part += q[2 * i + 1] * (float)((int)((c >> (16 + 4 * i)) & 15) - 8);
                    }
                }
                dot += part * __half2float(sc[g]);
            }
            x = dot * a.scale_log2;
        }
        float top = x;
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(m, top);
        if (mn == -INFINITY) continue;
        const float e = exp2f(x - mn), r = exp2f(m - mn);
        m = mn;
        sum = sum * r + e;
        for (int i = 0; i < 4; ++i) acc[i] *= r;
        const unsigned who = __ballot_sync(0xffffffffu, see);
        for (int k = 0; k < 32; ++k) {
            if (!((who >> k) & 1)) continue;
            const float pk = __shfl_sync(0xffffffffu, e, k);
            const uint64_t bk = __shfl_sync(0xffffffffu, (unsigned long long)blk, k);
            const int sk = (j0 + k) % ps;
            if (lane >= W * 2) continue;
            const uint8_t *base = reinterpret_cast<const uint8_t *>(bk);
            const uint32_t c = reinterpret_cast<const uint16_t *>(base + ps * (D / 2) + sk * (D / 2))[lane];
            const float s = __half2float(reinterpret_cast<const __half *>(base + ps * D)[ps * NG + sk * NG + lane % NG]);
            for (int i = 0; i < 4; ++i) acc[i] += pk * (s * (float)((int)((c >> (4 * i)) & 15) - 8));
        }
    }
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0 && a.lse)
        a.lse[row] = sum > 0.0f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    if (lane < W * 2) {
        const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
        const int d = 32 * (lane % NG) + 4 * (lane / NG);
        for (int i = 0; i < 4; ++i)
            a.out[(size_t)row * D + d + i] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i] * r));
    }
}

}  // namespace

cudaError_t launch_kv4_attn(const KvAttnArgs &a, int D, cudaStream_t s) {
    const long long rows = (long long)a.batch.tokens * a.q_heads;
    auto c = pdl_config((unsigned)((rows + 3) / 4), 128, 0, s);
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return D == 128 ? cudaLaunchKernelEx(&c, kv4_attn_kernel<128>, a)
                    : cudaLaunchKernelEx(&c, kv4_attn_kernel<64>, a);
}

}  // namespace moe
