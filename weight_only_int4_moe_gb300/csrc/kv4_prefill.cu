// Attention over the 4-bit cache for many query rows (include/moe_kv4.h): prompts,
// chunks and larger verify batches, where the products are the bound.
//
// An item is up to 256 query rows that share a kv head (its group's heads of
// consecutive tokens), two tiles of 128 for tcgen05.mma, against tiles of 128
// tokens.  Per tile of tokens and rows,
//   S = Q K^T   (128 x 128 x D, both operands fp16 in shared memory)
//   P = 2^(S - m) in fp16, written over S in tensor memory
//   O += P V    (128 x D x 128, P from tensor memory, V from shared memory)
// with the running maximum m and the sum of a row in the one thread that owns the
// row.  O is rescaled only when a row's maximum has grown by more than 2^8 since
// its last rescale (the probabilities then stay below 2^8, far inside fp16, and
// the quotient O / l does not depend on m).
//
// Roles of the 16 warps: two warpgroups each own one tile of rows (load its Q,
// softmax, output); one warpgroup turns codes into fp16 operand tiles, its loads
// one tile ahead in registers; one warp issues the MMAs, alternating between the
// two tiles of rows so that the softmax of one runs under the products of the
// other.  K tiles are K-major, V tiles are left in token order and read N-major;
// the order of V's columns is the order in which its codes unpack, undone when
// the output is written.
//
// The list of (request, row tile, kv head) items' token tiles is cut into equal
// runs, one a CTA; parts of an item are joined through the workspace by the last
// CTA to arrive, in list order.
#include "dequant.cuh"
#include "kv4_launch.cuh"

namespace moe {

namespace {

constexpr int kTok = 128;        // tokens of a unit
constexpr int kRowsItem = 256;
constexpr int kChunks = 1024;
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;
// Registers a thread of each role (multiples of 8): a row of S is 128 of them.  The
// four warpgroups' shares add up to what the block is launched with, 4 x 128.
constexpr int kRegsLaunch = 128, kRegsSoftmax = 168, kRegsCodes = 120, kRegsMma = 56;
static_assert(2 * kRegsSoftmax + kRegsCodes + kRegsMma == 4 * kRegsLaunch, "register shares");
static_assert(kThreads * kRegsLaunch == 65536, "the block takes the whole register file");

template <int D>
struct Cfg {
    static constexpr int NG = D / 32;
    static constexpr int kTileBytes = kTok * D * 2;   // an operand tile
    static constexpr int kQ = 0;                      // two tiles of rows
    static constexpr int kK = 2 * kTileBytes;         // two K tiles, two V tiles
    static constexpr int kV = 4 * kTileBytes;
    static constexpr int kSmem = 6 * kTileBytes + 1024;
    static constexpr int kPitch = D + 4;
    static constexpr int kSlot = kRowsItem * kPitch;
    static constexpr int kLoads = D == 128 ? 4 : 2;   // 16-byte loads a thread for K (and V)
};

enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kQFull = 8, kSFull = 10, kPFull = 12, kOFull = 14, kBars = 16 };

struct Shared {
    uint64_t bar[kBars];
    uint32_t tmem, warp_tot[kThreads / 32];
    int abort_flag, last_of;
    uint32_t ok[8];              // runs of 16 tokens that have a page, by tile
    uint32_t prefix[kChunks + 1];
    uint32_t part_u0[2], part_u1[2];
    int part_b[2], part_h[2], part_rt[2];
};

struct Request {
    int q0, m, first, end, rows, row_tiles;
};

MOE_DEV Request request_of(const KvAttnArgs &a, int b) {
    Request r;
    r.q0 = a.batch.cu_q[b];
    r.m = a.batch.cu_q[b + 1] - r.q0;
    const int len = a.batch.kv_len[b];
    r.first = len - r.m;
    r.end = (int)min((long long)len, (long long)a.batch.stride * a.pool.ps);
    r.rows = r.m * a.group;
    const bool mine = r.m > 0 && r.rows >= a.rows_lo && r.rows <= a.rows_hi;
    r.row_tiles = mine ? (r.rows + kRowsItem - 1) / kRowsItem : 0;
    return r;
}

// Token tiles of a row tile: [lo, lo + n).
MOE_DEV int tiles_of(const KvAttnArgs &a, const Request &r, int rt, int &lo) {
    const int i_lo = rt * kRowsItem / a.group;
    const int i_hi = (min(r.rows, (rt + 1) * kRowsItem) - 1) / a.group;
    const int hi = max(0, min(r.end, r.first + i_hi + 1));
    lo = (a.window > 0 ? max(0, r.first + i_lo - a.window + 1) : 0) / kTok;
    return max(1, (hi + kTok - 1) / kTok - lo);
}

// Units of a request, by a whole warp.
MOE_DEV uint32_t request_units(const KvAttnArgs &a, const Request &r) {
    uint32_t n = 0;
    int lo;
    for (int rt = threadIdx.x & 31; rt < r.row_tiles; rt += 32) n += tiles_of(a, r, rt, lo);
    return __reduce_add_sync(0xffffffffu, n) * a.pool.hkv;
}

// A run of one item's tiles that a CTA works on.  Every warp of every role walks
// the same list (whole-warp calls).
struct Segment {
    Request r;
    int b, rt, h, tile0, n;       // tile0: the first token tile of the run
    uint32_t i_u0, i_u1;
    int rows;                     // of the item
    bool whole;
};

struct Walk {
    uint32_t u, u_end, b_u0;
    int b, per_chunk;
    const uint32_t *prefix;

    MOE_DEV void start(const KvAttnArgs &a, const uint32_t *pre, int chunks, int per, uint32_t lo,
                       uint32_t hi) {
        u = lo;
        u_end = hi;
        prefix = pre;
        per_chunk = per;
        int x = 0, y = chunks - 1;
        while (x < y) {
            const int mid = (x + y + 1) >> 1;
            if (pre[mid] <= u)
                x = mid;
            else
                y = mid - 1;
        }
        b = x * per;
        b_u0 = pre[x];
    }

    MOE_DEV bool next(const KvAttnArgs &a, Segment &s) {
        if (u >= u_end) return false;
        s.r = request_of(a, b);
        while (true) {
            const uint32_t n = per_chunk == 1 ? prefix[b + 1] - prefix[b] : request_units(a, s.r);
            if (u < b_u0 + n) break;
            b_u0 += n;
            s.r = request_of(a, ++b);
        }
        // the row tile: 32 at a time
        const int lane = threadIdx.x & 31, hkv = a.pool.hkv;
        uint32_t at = u - b_u0, base = 0;
        for (int rt0 = 0;; rt0 += 32) {
            int lo = 0;
            const int rt = rt0 + lane;
            const uint32_t n = rt < s.r.row_tiles ? (uint32_t)tiles_of(a, s.r, rt, lo) : 0u;
            uint32_t x = n * hkv;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const unsigned who = __ballot_sync(0xffffffffu, at < base + x);
            if (!who) {
                base += __shfl_sync(0xffffffffu, x, 31);
                continue;
            }
            const int l = __ffs(who) - 1;
            s.rt = rt0 + l;
            const uint32_t tiles = __shfl_sync(0xffffffffu, n, l);
            const uint32_t rt_u0 = base + __shfl_sync(0xffffffffu, x, l) - tiles * hkv;
            s.h = (int)((at - rt_u0) / tiles);
            s.i_u0 = b_u0 + rt_u0 + s.h * tiles;
            s.i_u1 = s.i_u0 + tiles;
            s.tile0 = __shfl_sync(0xffffffffu, lo, l) + (int)(u - s.i_u0);
            break;
        }
        s.b = b;
        const uint32_t end = min(u_end, s.i_u1);
        s.n = (int)(end - u);
        s.whole = u == s.i_u0 && end == s.i_u1;
        s.rows = min(kRowsItem, s.r.rows - s.rt * kRowsItem);
        u = end;
        return true;
    }
};

MOE_DEV void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

MOE_DEV void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// Byte offset of 16-byte chunk c of row r in an operand tile: 128-byte-wide column
// blocks of 128 rows, chunks permuted by the row (the 128-byte swizzle).
MOE_DEV uint32_t tile_at(int r, int c) {
    return (uint32_t)((c >> 3) * (kTok * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// K-major operand (rows of 64 elements, 128-byte swizzle): see smem_desc_sw128.
// The N-major operand's 64-column blocks are kTok * 128 bytes apart (leading
// offset), its groups of eight tokens 1024 bytes (stride offset).
MOE_DEV uint64_t desc_n_major(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((kTok * 128) >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// S = Q K^T: D / 16 MMAs, operands in column blocks of 64 dimensions; then commits.
template <int D>
MOE_DEV void mma_qk(uint32_t d_tmem, uint32_t q, uint32_t k, uint32_t idesc) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const uint64_t qd = smem_desc_sw128(q + c * kTok * 128), kd = smem_desc_sw128(k + c * kTok * 128);
        asm volatile(
            "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
            "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
            "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
            "l"(qd), "l"(kd), "r"(idesc), "r"((uint32_t)c)
            : "memory");
    }
}

// O (+)= P V: kTok / 16 MMAs; P's columns advance by 8, V's tokens by 16 rows.
MOE_DEV void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
    for (int s = 0; s < kTok / 64; ++s) {
        const uint64_t vd = desc_n_major(v + s * 64 * 128);
        asm volatile(
            "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
            "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
            "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
            "add.u64 b1, %2, 128;\n\tadd.u64 b2, %2, 256;\n\tadd.u64 b3, %2, 384;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
            "r"(p_tmem + 32 * s), "l"(vd), "r"(idesc), "r"(s ? 1u : accumulate)
            : "memory");
    }
}

#define KV4_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), \
                     "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define KV4_P8(v, o) "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), \
                     "+r"(v[o + 5]), "+r"(v[o + 6]), "+r"(v[o + 7])

// 32 columns of the thread's lane, not waited for.
MOE_DEV void tmem_ld32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : KV4_R8(v, 0), KV4_R8(v, 8), KV4_R8(v, 16), KV4_R8(v, 24)
        : "r"(taddr)
        : "memory");
}
// Waits for the thread's loads; the registers of one pass through, so that no use
// of them can come before the wait (tmem_pass: for the further ones).
MOE_DEV void tmem_wait_ld(uint32_t *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : KV4_P8(v, 0), KV4_P8(v, 8), KV4_P8(v, 16), KV4_P8(v, 24)::"memory");
}
MOE_DEV void tmem_pass(uint32_t *v) {
    asm volatile("" : KV4_P8(v, 0), KV4_P8(v, 8), KV4_P8(v, 16), KV4_P8(v, 24)::"memory");
}

MOE_DEV float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

MOE_DEV uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
MOE_DEV void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
MOE_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
MOE_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A word's four nibble pairs as (q - 8) * s in fp16, exact (see dequant_row).
MOE_DEV void scaled_codes(uint32_t w, uint32_t s, uint32_t (&x)[4]) {
    const __half2 m24 = __hmul2(as_h2(s), as_h2(0xCE00CE00u));
    const uint32_t t[4] = {w << 6, w << 2, w >> 2, w >> 6};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = as_u32(__hfma2(as_h2((t[i] & 0x03C003C0u) | 0x4C004C00u), as_h2(s), m24));
}

// Codes and scales of a thread's part of one tile, on their way from global memory.
template <int D>
struct Packed {
    uint4 k[Cfg<D>::kLoads], v[Cfg<D>::kLoads];
    uint32_t ks[Cfg<D>::kLoads][D / 64], vs[Cfg<D>::kLoads][D / 64];
};

template <int N>
MOE_DEV void more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
MOE_DEV void fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const KvAttnArgs a) {
    using C = Cfg<D>;
    constexpr int NG = C::NG;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Shared sh;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, hkv = a.pool.hkv;
    pdl_wait();
    if (tid == 0) {
        sh.abort_flag = 0;
        const int counts[8] = {128, 1, 128, 1, 128, 1, 128, 1};
        for (int i = 0; i < kBars; ++i) mbar_init(smem_u32(&sh.bar[i]), counts[i / 2]);
        mbar_fence_init();
        sh.part_u0[0] = sh.part_u1[0] = sh.part_u0[1] = sh.part_u1[1] = 0;
    }
    if (w == 15) {
        tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
        tmem_relinquish();
    }
    // prefix of units over chunks of requests
    const int per_chunk = (a.batch.requests + kChunks - 1) / kChunks;
    const int chunks = (a.batch.requests + per_chunk - 1) / per_chunk;
    uint32_t carry = 0;
    for (int c0 = 0; c0 < chunks; c0 += kThreads) {
        uint32_t n = 0;
        for (int k = 0; k < per_chunk; ++k) {
            const int b = (c0 + tid) * per_chunk + k;
            Request r{};
            if (b < a.batch.requests) r = request_of(a, b);
            if (blockIdx.x == 0 && r.row_tiles && r.end < r.first + r.m)
                kv_report(a.err, MOE_KV4_DEVERR_PAGE);  // beyond its table
            // long requests' row tiles are counted by the warp together
            const bool big = r.row_tiles > 4;
            int lo;
            if (!big)
                for (int rt = 0; rt < r.row_tiles; ++rt) n += (uint32_t)tiles_of(a, r, rt, lo) * hkv;
            unsigned who = __ballot_sync(0xffffffffu, big);
            while (who) {
                const int l = __ffs(who) - 1;
                who &= who - 1;
                const int bb = __shfl_sync(0xffffffffu, b, l);
                const uint32_t x = request_units(a, request_of(a, bb));
                if (lane == l) n += x;
            }
        }
        uint32_t x = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) sh.warp_tot[w] = x;
        __syncthreads();
        uint32_t before = carry, all = carry;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < w) before += sh.warp_tot[i];
            all += sh.warp_tot[i];
        }
        if (c0 + tid < chunks) sh.prefix[c0 + tid] = before + x - n;
        carry = all;
        __syncthreads();
    }
    if (tid == 0) sh.prefix[chunks] = carry;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t total = carry;
    const uint32_t per = max((uint32_t)a.min_units, (total + gridDim.x - 1) / gridDim.x);
    const uint32_t c_lo = min(total, blockIdx.x * per), c_hi = min(total, c_lo + per);
    const uint32_t tmem = sh.tmem;
    const float sl2 = fmaxf(fabsf(a.scale_log2), 1e-30f);
    auto bar = [&](int i) { return smem_u32(&sh.bar[i]); };
    // S (and P over it) of the two row tiles, then their O
    auto s_col = [&](int m) { return tmem + 128u * m; };
    auto o_col = [&](int m) { return tmem + 256u + 128u * m; };
    int *abort_flag = &sh.abort_flag;

    if (c_lo < c_hi) {
        Walk walk;
        walk.start(a, sh.prefix, chunks, per_chunk, c_lo, c_hi);
        Segment sg;
        if (w < 8) {
            // ------------------------------------------- softmax of a tile of rows --
            more_regs<kRegsSoftmax>();
            const int m = w >> 2, r = tid & 127;  // the thread's row in its tile
            const uint32_t lane_off = (uint32_t)(32 * (w & 3)) << 16;
            const uint32_t s_at = s_col(m) + lane_off, o_at = o_col(m) + lane_off;
            uint32_t s_ph = 0, o_ph = 0, tiles = 0;
            while (walk.next(a, sg)) {
                if (m * 128 >= sg.rows) {
                    tiles += sg.n;
                    continue;
                }
                // Q: 16-byte chunks of the tile's rows, converted and swizzled
                const int row_base = sg.rt * kRowsItem + m * 128, n_rows = min(128, sg.rows - m * 128);
                bool bad = false;
                const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
                for (int c = r; c < 128 * (D / 8); c += 128) {
                    const int qr = c / (D / 8), ch = c % (D / 8);
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (qr < n_rows) {
                        const int i = (row_base + qr) / a.group, hh = row_base + qr - i * a.group;
                        v = *reinterpret_cast<const uint4 *>(a.q + (size_t)(sg.r.q0 + i) * a.q_stride +
                                                             (size_t)(sg.h * a.group + hh) * D + 8 * ch);
                    }
                    v = bf16x8_to_f16x8_sat(v, bad);
                    sts128(smem + C::kQ + m * C::kTileBytes + tile_at(qr, ch), v.x ^ flip, v.y ^ flip,
                           v.z ^ flip, v.w ^ flip);
                }
                if (__any_sync(0xffffffffu, bad) && lane == 0) kv_report(a.err, MOE_KV4_DEVERR_RANGE);
                fence_proxy_async_shared();
                mbar_arrive(bar(kQFull + m));

                const int i = (row_base + r) / a.group, hh = row_base + r - i * a.group;
                const bool live = r < n_rows;
                const int p = sg.r.first + i;
                const int hi = live ? min(p, sg.r.end - 1) : -1;
                const int lo = a.window > 0 ? p - a.window : -1;
                const uint64_t word = a.tree && live ? a.tree[sg.r.q0 + i] : 0;
                // tokens that every row of the warp sees
                const int open = __reduce_min_sync(0xffffffffu, live ? (a.tree ? min(hi + 1, sg.r.first) : hi + 1)
                                                                     : INT32_MAX);
                const int shut = __reduce_max_sync(0xffffffffu, live ? lo + 1 : 0);
                const bool any_live = __any_sync(0xffffffffu, live);
                float top = -INFINITY, sum = 0.0f;
                bool gave_up = false;
                for (int k = 0; k < sg.n; ++k) {
                    const bool ok_wait = mbar_wait(bar(kSFull + m), s_ph, abort_flag, a.err);
                    s_ph ^= 1;
                    if (__any_sync(0xffffffffu, !ok_wait)) {
                        gave_up = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ok = sh.ok[tiles & 7];
                    ++tiles;
                    uint32_t s[128];
                    if (any_live) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, s + 32 * c);
                        tmem_wait_ld(s);
                        tmem_pass(s + 32);
                        tmem_pass(s + 64);
                        tmem_pass(s + 96);
                        const int j0 = (sg.tile0 + k) * kTok;
                        if (ok != 0xFFu || j0 + kTok > open || j0 < shut) {
#pragma unroll
                            for (int c = 0; c < 128; ++c) {
                                const int j = j0 + c;
                                bool see = j <= hi && j > lo && ((ok >> (c / 16)) & 1u);
                                if (a.tree && j >= sg.r.first)
                                    see = see && j - sg.r.first < 64 && ((word >> (j - sg.r.first)) & 1u);
                                if (!see) s[c] = 0xff800000u;  // -inf
                            }
                        }
                        float mx[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(s[c]);
#pragma unroll
                        for (int c = 4; c < 128; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(s[c]));
                        const float now = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        // the first maximum of a run is taken as it is; later ones only when
                        // they have grown by more than 2^8
                        const bool grow = now > top && (top == -INFINITY || (now - top) * sl2 > 8.0f);
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? ex2((top - now) * sl2) : 1.0f;
                            if (grow) top = now;
                            sum *= f;
                            if (k > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
                                for (int c = 0; c < D / 16; ++c) {
                                    float o[16];
                                    tmem_ld_32x32b_x16_wait(o_at + 16 * c, o);
                                    asm volatile(
                                        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, "
                                        "%5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
                                            o_at + 16 * c),
                                        "f"(o[0] * f), "f"(o[1] * f), "f"(o[2] * f), "f"(o[3] * f),
                                        "f"(o[4] * f), "f"(o[5] * f), "f"(o[6] * f), "f"(o[7] * f),
                                        "f"(o[8] * f), "f"(o[9] * f), "f"(o[10] * f), "f"(o[11] * f),
                                        "f"(o[12] * f), "f"(o[13] * f), "f"(o[14] * f), "f"(o[15] * f)
                                        : "memory");
                                }
                            }
                        }
                        const float off = top == -INFINITY ? 0.0f : -top * sl2;
                        const uint64_t sc2 = pack2(sl2, sl2), off2 = pack2(off, off);
                        uint64_t sum2[2] = {pack2(sum, 0.0f), 0};
#pragma unroll
                        for (int c = 0; c < 128; c += 2) {
                            float x, y;
                            unpack2(fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, off2),
                                    x, y);
                            x = ex2(x);
                            y = ex2(y);
                            sum2[(c >> 1) & 1] = add2(sum2[(c >> 1) & 1], pack2(x, y));
                            s[c / 2] = as_u32(__floats2half2_rn(x, y));
                        }
                        float x, y;
                        unpack2(add2(sum2[0], sum2[1]), x, y);
                        sum = x + y;
                        uint32_t *s2 = s;
                        tmem_st_32x32b_x32(s_at, *reinterpret_cast<const uint32_t(*)[32]>(s2));
                        tmem_st_32x32b_x32(s_at + 32, *reinterpret_cast<const uint32_t(*)[32]>(s2 + 32));
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(bar(kPFull + m));
                }
                if (gave_up) break;
                // O of the run
                const bool ok_wait = mbar_wait(bar(kOFull + m), o_ph, abort_flag, a.err);
                o_ph ^= 1;
                if (__any_sync(0xffffffffu, !ok_wait)) break;
                tc_fence_after();
                if (any_live) {
                    const float inv = sg.whole ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
                    const size_t o_row = (size_t)(sg.r.q0 + i) * a.q_heads + sg.h * a.group + hh;
                    const int part = sg.i_u0 > c_lo ? 1 : 0;
                    float *slot = a.cta_slots + ((size_t)2 * blockIdx.x + part) * C::kSlot +
                                  (m * 128 + r) * C::kPitch;
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        // columns of four V pieces g = 4a..: two groups' 16 dimensions
                        uint32_t o[32];
                        tmem_ld32(o_at + 32 * q, o);
                        tmem_wait_ld(o);
                        const int pp = q >> 1, d0 = 64 * pp + 16 * (q & 1);
                        if (!live) continue;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float x[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                x[e] = __uint_as_float(o[(e >> 2) * 8 + 2 * (e & 3) + half]) * inv;
                            if (sg.whole) {
                                uint32_t y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const __nv_bfloat162 z = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                                    y[e] = *reinterpret_cast<const uint32_t *>(&z);
                                }
                                uint4 *dst = reinterpret_cast<uint4 *>(a.out + o_row * D + d0 + 32 * half);
                                dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                                dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                            } else {
                                float4 *dst = reinterpret_cast<float4 *>(slot + d0 + 32 * half);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                            }
                        }
                    }
                    if (live) {
                        if (!sg.whole) {
                            slot[D] = top;
                            slot[D + 1] = sum;
                        } else if (a.lse) {
                            a.lse[o_row] = sum > 0.0f ? (top * sl2 + log2f(sum)) * 0.6931471805599453f
                                                      : -INFINITY;
                        }
                    }
                }
                if (!sg.whole && tid == 0) {
                    const int part = sg.i_u0 > c_lo ? 1 : 0;
                    sh.part_u0[part] = sg.i_u0;
                    sh.part_u1[part] = sg.i_u1;
                    sh.part_b[part] = sg.b;
                    sh.part_h[part] = sg.h;
                    sh.part_rt[part] = sg.rt;
                }
                tc_fence_before();  // the reads of O before the next run's first product
            }
            fewer_regs<kRegsLaunch>();
        } else if (w < 12) {
            // ----------------------------------------------- codes to operand tiles --
            fewer_regs<kRegsCodes>();
            constexpr int kLanesRow = D == 128 ? 4 : 2;         // 16-byte chunks of a row
            constexpr int kStep = 128 / kLanesRow;              // rows of one load of the group
            const int dt = tid - 256, row_l = dt / kLanesRow, ch = dt % kLanesRow;
            const int ps = a.pool.ps;
            Ring kr(2), vr(2);
            uint32_t tiles = 0;
            bool gave_up = false;
            while (!gave_up && walk.next(a, sg)) {
                const int32_t *table = a.batch.tables + (size_t)sg.b * a.batch.stride;
                const int ppt = kTok / ps;
                int e_base = 0, ids = -1;
                auto load_ids = [&](int from) {
                    e_base = from;
                    const int e = from + lane;
                    ids = -1;
                    if (e < (sg.tile0 + sg.n) * ppt && (long long)e * ps < sg.r.end) {
                        ids = table[e];
                        if ((unsigned)ids >= (unsigned)a.pool.n_pages) {
                            ids = -1;
                            if (sg.h == 0 && w == 8) kv_report(a.err, MOE_KV4_DEVERR_PAGE);
                        }
                    }
                };
                load_ids(sg.tile0 * ppt);
                Packed<D> pk;
                uint32_t ok_next = 0;
                // requests the k-th tile's K (or V) part of this thread
                auto load = [&](int k, bool key) {
                    const int e0 = (sg.tile0 + k) * ppt;
                    if (key && e0 + ppt > e_base + 32) load_ids(e0);
                    if (key) {
                        uint32_t ok = 0;
                        for (int i = 0; i < ppt; ++i)
                            if (__shfl_sync(0xffffffffu, ids, e0 - e_base + i) >= 0)
                                ok |= ((1u << (ps / 16)) - 1u) << (i * (ps / 16));
                        ok_next = ok;
                    }
#pragma unroll
                    for (int i = 0; i < C::kLoads; ++i) {
                        const int row = i * kStep + row_l;
                        const int id = __shfl_sync(0xffffffffu, ids, e0 - e_base + row / ps);
                        const bool live = id >= 0 && (sg.tile0 + k) * kTok + row < sg.r.end;
                        const int slot = row & (ps - 1);
                        const uint8_t *blk = kv_block(a.pool, live ? id : 0, sg.h);
                        const uint8_t *code = blk + (key ? 0 : ps * (D / 2)) + slot * (D / 2) + 16 * ch;
                        const uint32_t *sc = reinterpret_cast<const uint32_t *>(
                            blk + ps * D + (key ? 0 : ps * (NG * 2)) + slot * (NG * 2));
                        uint4 c = make_uint4(0, 0, 0, 0);
                        uint32_t z[D / 64];
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) z[x] = 0;
                        if (live) {
                            c = *reinterpret_cast<const uint4 *>(code);
#pragma unroll
                            for (int x = 0; x < D / 64; ++x) z[x] = sc[x];
                        }
                        (key ? pk.k[i] : pk.v[i]) = c;
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) (key ? pk.ks[i][x] : pk.vs[i][x]) = z[x];
                    }
                };
                load(0, true);
                load(0, false);
                for (int k = 0; k < sg.n; ++k) {
                    // K: the chunk's words are (t, G) for its t's; a word is dimensions
                    // 32G + 8t.., the row's 16-byte chunk 4G + t
                    if (__any_sync(0xffffffffu,
                                   !mbar_wait(bar(kKEmpty + kr.idx), kr.ph ^ 1, abort_flag, a.err))) {
                        gave_up = true;
                        break;
                    }
                    if (dt == 0) sh.ok[tiles & 7] = ok_next;
                    ++tiles;
                    const uint32_t kd = smem + C::kK + kr.idx * C::kTileBytes;
#pragma unroll
                    for (int i = 0; i < C::kLoads; ++i) {
                        const int row = i * kStep + row_l;
                        const uint32_t words[4] = {pk.k[i].x, pk.k[i].y, pk.k[i].z, pk.k[i].w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int G = D == 128 ? u : u & 1, t = D == 128 ? ch : 2 * ch + (u >> 1);
                            const uint32_t s = __byte_perm(pk.ks[i][G / 2], 0, G & 1 ? 0x3232 : 0x1010);
                            uint32_t x[4];
                            scaled_codes(words[u], s, x);
                            sts128(kd + tile_at(row, 4 * G + t), x[0], x[1], x[2], x[3]);
                        }
                    }
                    fence_proxy_async_shared();
                    mbar_arrive(bar(kKFull + kr.idx));
                    kr.next();
                    if (k + 1 < sg.n) load(k + 1, true);
                    // V: a word is piece g of groups 2p and 2p + 1, column chunk 8p + g
                    if (__any_sync(0xffffffffu,
                                   !mbar_wait(bar(kVEmpty + vr.idx), vr.ph ^ 1, abort_flag, a.err))) {
                        gave_up = true;
                        break;
                    }
                    const uint32_t vd = smem + C::kV + vr.idx * C::kTileBytes;
#pragma unroll
                    for (int i = 0; i < C::kLoads; ++i) {
                        const int row = i * kStep + row_l;
                        const uint32_t words[4] = {pk.v[i].x, pk.v[i].y, pk.v[i].z, pk.v[i].w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int pp = D == 128 ? u & 1 : 0, g = D == 128 ? 2 * ch + (u >> 1) : 4 * ch + u;
                            uint32_t x[4];
                            scaled_codes(words[u], pk.vs[i][pp], x);
                            sts128(vd + tile_at(row, 8 * pp + g), x[0], x[1], x[2], x[3]);
                        }
                    }
                    fence_proxy_async_shared();
                    mbar_arrive(bar(kVFull + vr.idx));
                    vr.next();
                    if (k + 1 < sg.n) load(k + 1, false);
                }
            }
            more_regs<kRegsLaunch>();
        } else {
            fewer_regs<kRegsMma>();
            // ----------------------------------------------------------------- MMAs --
            const uint32_t id_s = idesc_f16_m128(kTok);
            const uint32_t id_o = idesc_f16_m128(D) | (1u << 16);  // B N-major
            Ring kr(2), vr(2);
            uint32_t p_ph[2] = {0, 0}, q_ph[2] = {0, 0};
            bool gave_up = false;
            auto wait = [&](int b, uint32_t ph) {
                if (__any_sync(0xffffffffu, !mbar_wait(bar(b), ph, abort_flag, a.err))) gave_up = true;
                tc_fence_after();
                return !gave_up;
            };
            while (w == 12 && !gave_up && walk.next(a, sg)) {
                const int nm = sg.rows > 128 ? 2 : 1;
                for (int m = 0; m < nm; ++m) {
                    if (!wait(kQFull + m, q_ph[m])) break;
                    q_ph[m] ^= 1;
                }
                if (gave_up || !wait(kKFull + kr.idx, kr.ph)) break;
                for (int m = 0; m < nm; ++m) {
                    mma_qk<D>(s_col(m), smem + C::kQ + m * C::kTileBytes,
                              smem + C::kK + kr.idx * C::kTileBytes, id_s);
                    tc_commit2_elect(bar(kSFull + m), m == nm - 1 ? bar(kKEmpty + kr.idx) : 0u);
                }
                kr.next();
                for (int k = 0; k < sg.n && !gave_up; ++k) {
                    if (!wait(kVFull + vr.idx, vr.ph)) break;
                    for (int m = 0; m < nm; ++m) {
                        if (!wait(kPFull + m, p_ph[m])) break;
                        p_ph[m] ^= 1;
                        mma_pv(o_col(m), s_col(m), smem + C::kV + vr.idx * C::kTileBytes, id_o, k > 0);
                        tc_commit2_elect(k == sg.n - 1 ? bar(kOFull + m) : 0u,
                                         m == nm - 1 ? bar(kVEmpty + vr.idx) : 0u);
                        if (k + 1 < sg.n) {
                            if (m == 0 && !wait(kKFull + kr.idx, kr.ph)) break;
                            mma_qk<D>(s_col(m), smem + C::kQ + m * C::kTileBytes,
                                      smem + C::kK + kr.idx * C::kTileBytes, id_s);
                            tc_commit2_elect(bar(kSFull + m), m == nm - 1 ? bar(kKEmpty + kr.idx) : 0u);
                        }
                    }
                    vr.next();
                    if (k + 1 < sg.n) kr.next();
                }
            }
            more_regs<kRegsLaunch>();
        }
    }
    tc_fence_before();
    __threadfence();
    __syncthreads();
    tc_fence_after();
    if (w == 15) tmem_dealloc(tmem, kTmemCols);

    // items shared with other CTAs: the last of them adds the parts up
    constexpr int kQuads = D / 4;
    for (int part = 0; part < 2; ++part) {
        const uint32_t u0 = sh.part_u0[part], u1 = sh.part_u1[part];
        if (u0 == u1) continue;
        const uint32_t c0 = u0 / per, c1 = (u1 - 1) / per;
        if (tid == 0) {
            const int old = atomicAdd(a.counters + c0, 1);
            sh.last_of = old == (int)(c1 - c0);
            if (sh.last_of) a.counters[c0] = 0;
        }
        __syncthreads();
        const bool mine = sh.last_of;
        __syncthreads();
        if (!mine) continue;
        __threadfence();
        const Request rq = request_of(a, sh.part_b[part]);
        const int rt = sh.part_rt[part], h = sh.part_h[part];
        const int rows = min(kRowsItem, rq.rows - rt * kRowsItem);
        for (int e = tid; e < rows * kQuads; e += kThreads) {
            const int row = e / kQuads, d4 = e % kQuads;
            float mm = -INFINITY, ll = 0.0f;
            float4 s = make_float4(0, 0, 0, 0);
            for (uint32_t c = c0; c <= c1; ++c) {
                const float *pr = a.cta_slots +
                                  ((size_t)2 * c + (c == c0 && u0 > c0 * per ? 1 : 0)) * C::kSlot +
                                  row * C::kPitch;
                const float pm = pr[D], pl = pr[D + 1];
                const float4 v = *reinterpret_cast<const float4 *>(pr + 4 * d4);
                const float nm = fmaxf(mm, pm);
                const float x = mm > -INFINITY ? ex2((mm - nm) * sl2) : 0.0f;
                const float y = pm > -INFINITY ? ex2((pm - nm) * sl2) : 0.0f;
                mm = nm;
                ll = ll * x + pl * y;
                s.x = s.x * x + v.x * y;
                s.y = s.y * x + v.y * y;
                s.z = s.z * x + v.z * y;
                s.w = s.w * x + v.w * y;
            }
            const int rr = rt * kRowsItem + row, i = rr / a.group, hh = rr - i * a.group;
            const size_t o = (size_t)(rq.q0 + i) * a.q_heads + h * a.group + hh;
            const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x * inv, s.y * inv);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(s.z * inv, s.w * inv);
            *reinterpret_cast<uint2 *>(a.out + o * D + 4 * d4) = make_uint2(
                *reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            if (a.lse && d4 == 0)
                a.lse[o] = ll > 0.0f ? (mm * sl2 + log2f(ll)) * 0.6931471805599453f : -INFINITY;
        }
    }
}

template <int D>
cudaError_t launch(const KvAttnArgs &a, int grid, cudaStream_t s) {
    static bool set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(kv4_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) set[dev] = true;
    }
    auto c = pdl_config((unsigned)grid, kThreads, Cfg<D>::kSmem, s);
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return cudaLaunchKernelEx(&c, kv4_prefill_kernel<D>, a);
}

}  // namespace

size_t kv4_prefill_slot_bytes(int D, int ctas) {
    return (size_t)ctas * 2 * kRowsItem * (D + 4) * 4;
}

cudaError_t launch_kv4_prefill(KvAttnArgs a, int D, void *slots, int ctas, cudaStream_t s) {
    a.cta_slots = reinterpret_cast<float *>(slots);
    a.min_units = 2;
    return D == 128 ? launch<128>(a, ctas, s) : launch<64>(a, ctas, s);
}

}  // namespace moe
