// Attention over the 4-bit cache for few query rows (include/moe_kv4.h): decode
// and small verify batches, where the cache's bytes are the bound.
//
// The query rows that share a kv head (its group's heads of all new tokens) are
// taken 8 NT at a time against tiles of 64 tokens.  The transposed products put
// tokens, then head dimensions, on the 16-high side of mma.m16n8k16 and the few
// rows on its 8-wide side, so that no instruction works on padding:
//   S^T[token, row] = K Q^T        O^T[dim, row] = V^T P^T
// The column of an accumulator is a row of the query in both, so the running
// maximum and the rescaling need no exchange between the two products.
//
// Codes become operands without leaving the lane that loads them.  A K word holds
// eight dimensions of one group for one token: masked and ORed with an fp16
// exponent they are four operand registers.  With one row tile the group's scale
// multiplies the group's fp32 partial score (four FMAs per 16 tokens and group
// instead of eight fp16 ones), the operands are 64 + q and the accumulator starts
// at -72 sum(q); with two the operands are (q - 8) scale, exact in fp16, as for the
// expert weights.  What cancels against the -72 sum(q) costs the fp32 scores about three
// bits, which leaves them inside the bound of a sum of D fp32 terms (D 2^-23 of their
// magnitudes, tested with keys of few large codes); operands q - 8, a subtraction more
// each, would keep the bits at 93 and 69 us below.  V pieces of two tokens are
// interleaved by one byte permute into (token, token + 1) pairs and take their two scales
// by the same exact FMA.
//
// Work is cut by tokens: all (request, row tile, kv head) items' tiles in one
// list, every CTA an equal run of it, every warp of the CTA an equal part of the
// run with a ring of tiles of its own, filled by bulk copies (a tile of a page
// size of 64 is one contiguous block).  Warps of a CTA join their parts of an item
// through shared memory, CTAs through the workspace, the last one to arrive adding
// them up in list order.
//
// Measured: 90 streams of up to 8192 tokens, 56 heads over 8 kv heads of 128: 89 us,
// 4.6 TB/s of the 6.8 that a copy reaches; two of 131071 tokens, 64 heads: 66 us, the same
// rate; one of 777, 32 heads: 12 us.  Bound by latency, not bytes and not yet by a pipe: a
// tile of 64 tokens is some 1000 instructions of a warp, most of them the unpacking, in
// one chain of products, softmax and products, and with the three warps a scheduler that
// the registers allow the issue slots are 58 % busy, the ALU pipe 45 %, FMA 33 %, tensor
// 23 %.  Joining the parts is a tenth of the time on the ragged batch.  Half tiles (half the code and the score registers) were slower:
// 95 and 71 us.  12 warps for 8 rows, 8 for 16: what the registers allow.
#include <atomic>

#include "dequant.cuh"
#include "kv4_launch.cuh"

namespace moe {

namespace {

constexpr int kTile = 64;       // tokens of a unit of work
constexpr int kChunks = 1024;   // entries of the prefix table over requests
// Units before an item's first tile that hold no work: what a warp spends on a new
// item (its queries, the first copies' latency), in tiles.
constexpr int kPad = 1;


template <int D, int NT>
struct Cfg {
    static constexpr int NG = D / 32;
    static constexpr int kTileBytes = kTile * (D + D / 8);
    static constexpr int kStages = D == 128 ? 2 : 3;
    static constexpr int kWarps = NT == 1 ? 12 : 8;
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = D + 4;                   // floats of a partial's row
    static constexpr int kSlot = kRows * kPitch;           // D sums, then m and l
    static constexpr int kRing = kStages * kTileBytes;
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kSlot * 4 <= kRing, "a warp's last partial reuses its ring");
};

struct Meta {        // where a warp's partial belongs
    uint32_t u0, u1; // the item's tiles as units; u0 == u1: none
    int q0, rows, h, row0; // the request's first token; the item's rows from row0 on
};

MOE_DEV void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// The same with an accumulator to start from that stays as it is.
MOE_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                      uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

MOE_DEV void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                      uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

MOE_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

MOE_DEV uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <int N>
MOE_DEV void lds_words(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = lds128(addr);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    } else {
        w[0] = lds32(addr);
    }
}

// The four nibble pairs of a word as fp16 pairs 64 + q.
MOE_DEV void codes64(uint32_t w, const KvConsts &k, uint32_t (&x)[4]) {
    const uint32_t v = w >> 8;
    x[0] = ((w * k.c16) & k.nib4) | k.magic64;
    x[1] = (w & k.nib4) | k.magic64;
    x[2] = ((v * k.c16) & k.nib4) | k.magic64;
    x[3] = (v & k.nib4) | k.magic64;
}

// The pairs of words lo and hi (their low two nibbles each) as (q - 8) * s, exact:
// (16 + q) * s - 24 * s.
MOE_DEV void codes_scaled(uint32_t lo, uint32_t hi, const KvConsts &k, uint32_t s, uint32_t (&x)[4]) {
    const __half2 m24 = __hmul2(as_h2(s), as_h2(k.cm24));
    const uint32_t t[4] = {lo * k.c64, lo * k.c4, hi * k.c64, hi * k.c4};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = as_u32(__hfma2(as_h2((t[i] & k.nib6) | k.magic16), as_h2(s), m24));
}

// What a request adds to the list of units.
struct Request {
    int q0, m, first, end, tile0, tiles, row_tiles;
};

MOE_DEV Request request_of(const KvAttnArgs &a, int q0, int q1, int len, int rows) {
    Request r;
    r.q0 = q0;
    r.m = q1 - q0;
    r.first = len - r.m;
    r.end = (int)min((long long)min(len, kKvMaxLen), (long long)a.batch.stride * a.pool.ps);
    const int start = a.window > 0 ? max(0, r.first - a.window + 1) : 0;
    r.tile0 = start / kTile;
    r.tiles = max(1, (r.end + kTile - 1) / kTile - r.tile0);
    // (a row range outside the batch's tokens is no request; compared before r.m is used,
    // as the difference of two ints may wrap)
    const bool mine = q0 >= 0 && q1 > q0 && q1 <= a.batch.tokens && r.m * a.group >= a.rows_lo &&
                      r.m * a.group <= a.rows_hi;
    r.row_tiles = mine ? (r.m * a.group + rows - 1) / rows : 0;
    return r;
}

MOE_DEV uint32_t units_of(const Request &r, int hkv) {
    return (uint32_t)(r.tiles + kPad) * (uint32_t)r.row_tiles * (uint32_t)hkv;
}

template <int D, int NT, int PS>
__global__ void __launch_bounds__(Cfg<D, NT>::kWarps * 32, 1)
    kv4_decode_kernel(const KvAttnArgs a) {
    using C = Cfg<D, NT>;
    constexpr int NG = C::NG, W = C::kWarps, S = C::kStages, RB = D / 2;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint32_t prefix[kChunks + 1];
    __shared__ uint64_t bars[W * S];
    __shared__ Meta meta[2 * W];
    __shared__ int run_of[2 * W + 1], n_runs, abort_flag, last_of[2];
    __shared__ uint32_t warp_tot[W];
    // Beside the prefill kernel nothing here depends on it, and what came before it is
    // complete (its blocks let this kernel start after their own wait): the wait moves to
    // the end, so that whatever follows finds both complete.
    if (!a.beside) pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
    const int hkv = a.pool.hkv, G = a.group;
    constexpr int ps = PS, ppt = kTile / PS;          // pages of a tile
    constexpr uint32_t kBlock = PS * (D + D / 8);     // bytes of a page of a head
    const float sl2 = a.sl2;
    if (tid == 0) abort_flag = 0;
    if (lane == 0)
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(&bars[w * S + s]), 1);
    mbar_fence_init();
    if (lane < 2) meta[2 * w + lane].u0 = meta[2 * w + lane].u1 = 0;

    // Units before each request.  Up to 32 requests: a lane of every warp holds one.
    // More: a prefix table over chunks of requests in shared memory.
    const bool few = a.batch.requests <= 32;
    int my_q0 = 0, my_q1 = 0, my_len = 0;
    uint32_t my_end = 0, total;
    const int per_chunk = (a.batch.requests + kChunks - 1) / kChunks;
    const int chunks = (a.batch.requests + per_chunk - 1) / per_chunk;
    auto load_request = [&](int b) {
        return request_of(a, a.batch.cu_q[b], a.batch.cu_q[b + 1], a.batch.kv_len[b], C::kRows);
    };
    auto check = [&](const Request &r) {
        if (blockIdx.x == 0 && r.row_tiles && r.end < r.first + r.m)
            kv_report(a.err, MOE_KV4_DEVERR_PAGE);  // beyond its table
    };
    if (few) {
        uint32_t n = 0;
        if (lane < a.batch.requests) {
            my_q0 = a.batch.cu_q[lane];
            my_q1 = a.batch.cu_q[lane + 1];
            my_len = a.batch.kv_len[lane];
            const Request r = request_of(a, my_q0, my_q1, my_len, C::kRows);
            n = units_of(r, hkv);
            if (w == 0) check(r);
        }
        my_end = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, my_end, d);
            if (lane >= d) my_end += y;
        }
        total = __shfl_sync(0xffffffffu, my_end, 31);
        __syncthreads();  // the barriers and flags set above
    } else {
        uint32_t carry = 0;
        for (int c0 = 0; c0 < chunks; c0 += W * 32) {
            uint32_t n = 0;
            if (c0 + tid < chunks)
                for (int b = (c0 + tid) * per_chunk;
                     b < min(a.batch.requests, (c0 + tid + 1) * per_chunk); ++b) {
                    const Request r = load_request(b);
                    n += units_of(r, hkv);
                    check(r);
                }
            uint32_t x = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (lane == 31) warp_tot[w] = x;
            __syncthreads();
            uint32_t before = carry, all = carry;
            for (int i = 0; i < W; ++i) {
                if (i < w) before += warp_tot[i];
                all += warp_tot[i];
            }
            if (c0 + tid < chunks) prefix[c0 + tid] = before + x - n;
            carry = all;
            __syncthreads();
        }
        if (tid == 0) prefix[chunks] = carry;
        __syncthreads();
        total = carry;
    }
    auto get_request = [&](int b) {
        if (!few) return load_request(b);
        return request_of(a, __shfl_sync(0xffffffffu, my_q0, b), __shfl_sync(0xffffffffu, my_q1, b),
                          __shfl_sync(0xffffffffu, my_len, b), C::kRows);
    };
    const uint32_t per = max((uint32_t)a.min_units, (total + gridDim.x - 1) / gridDim.x);
    const uint32_t c_lo = min(total, blockIdx.x * per), c_hi = min(total, c_lo + per);
    if (c_lo >= c_hi) {
        if (a.beside) pdl_wait();
        return;
    }
    // The warps' shares: one unit each to the first ones, or equal parts to all, so that
    // an item's tiles always lie in neighbouring warps.
    const uint32_t n_units = c_hi - c_lo;
    auto share = [&](uint32_t i) {
        return c_lo + (n_units < W ? min(i, n_units) : (uint32_t)((unsigned long long)n_units * i / W));
    };
    uint32_t u = share(w);
    const uint32_t u_end = share(w + 1);

    const uint32_t my_ring = smem_u32(ring) + w * C::kRing;
    const uint32_t my_bar = smem_u32(&bars[w * S]);
    Ring cons(S);
    const int tau = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;  // token of accumulator row g
    float *warp_slot = a.warp_slots + ((size_t)blockIdx.x * W + w) * C::kSlot;

    // the request that holds unit u
    int b = 0;
    uint32_t b_u0 = 0;
    if (u < u_end) {
        if (few) {
            b = __ffs(__ballot_sync(0xffffffffu, u < my_end)) - 1;
            if (b) b_u0 = __shfl_sync(0xffffffffu, my_end, b - 1);
        } else {
            int lo = 0, hi = chunks - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] <= u)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            b = lo * per_chunk;
            b_u0 = prefix[lo];
        }
    }
    bool aborted = false;
    while (u < u_end && !aborted) {
        Request rq = get_request(b);
        uint32_t n_b = units_of(rq, hkv);
        while (u >= b_u0 + n_b && b + 1 < a.batch.requests) {
            b_u0 += n_b;
            rq = get_request(++b);
            n_b = units_of(rq, hkv);
        }
        if (u >= b_u0 + n_b) break;  // the lengths changed under the call
        const uint32_t span = rq.tiles + kPad, item = (u - b_u0) / span;
        const uint32_t i_u0 = b_u0 + item * span + kPad, i_u1 = i_u0 + rq.tiles;  // its tiles
        u = max(u, i_u0);
        if (u >= u_end) break;
        const int h = item % hkv, rt = item / hkv;
        const uint32_t seg_end = min(u_end, i_u1);
        const int tile_lo = rq.tile0 + (int)(u - i_u0), n_tiles = (int)(seg_end - u);
        const int row0 = rt * C::kRows, rows = min(C::kRows, rq.m * G - row0);
        const int32_t *table = a.batch.tables + (size_t)b * a.batch.stride;

        // requested before the first tiles, behind which the queries would wait
        uint4 q_raw[NT][NG];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g, i = div_group(row0 + r, a.gdiv), hh = (row0 + r) - i * G;
            const uint16_t *src =
                a.q + (size_t)(rq.q0 + i) * a.q_stride + (size_t)(h * G + hh) * D + 8 * t;
#pragma unroll
            for (int G4 = 0; G4 < NG; ++G4) {
                q_raw[n][G4] = make_uint4(0, 0, 0, 0);
                if (r < rows) q_raw[n][G4] = *reinterpret_cast<const uint4 *>(src + 32 * G4);
            }
        }

        const uint8_t *head_base = a.pool.base + (size_t)h * kBlock;
        const size_t page_bytes = (size_t)hkv * kBlock;
        // page ids of the next tiles: lane l holds table entry e_base + l
        int e_base = tile_lo * ppt, ids = -1;
        auto load_ids = [&](int from) {
            e_base = from;
            const int e = from + lane;
            ids = -1;
            // (not the pages that the window of the item's first row has left behind: they
            // may be gone, or hold anything)
            const int seen = a.window > 0 ? rq.first + div_group(row0, a.gdiv) - a.window + 1 : 0;
            if (e < (tile_lo + n_tiles) * ppt && (long long)e * ps < rq.end &&
                (long long)(e + 1) * ps > seen) {
                ids = table[e];
                if ((unsigned)ids >= (unsigned)a.pool.n_pages) {
                    ids = -1;
                    if (h == 0 && rt == 0) kv_report(a.err, MOE_KV4_DEVERR_PAGE);
                }
            }
        };
        load_ids(e_base);
        // starts the copies of the segment's k-th tile; returns which of its four
        // runs of 16 tokens have a page
        auto fetch = [&](int k, uint32_t slot) -> uint32_t {
            const int e = (tile_lo + k) * ppt;
            if (e + ppt > e_base + 32) load_ids(e);
            uint32_t ok = 0, have = 0;
            int mine = -1;  // lane l < ppt copies the tile's page l
#pragma unroll
            for (int i = 0; i < ppt; ++i) {
                const int id = __shfl_sync(0xffffffffu, ids, e - e_base + i);
                if (id >= 0) {
                    ok |= ((1u << (ps / 16)) - 1u) << (i * (ps / 16));
                    ++have;
                }
                if (lane == i) mine = id;
            }
            if (lane == 0) mbar_arrive_expect_tx(my_bar + 8 * slot, have * kBlock);
            if (ppt > 1) __syncwarp();
            if (kDebugBounds && k == a.skip_tile && blockIdx.x == 0 && w == 0) mine = -1;
            if (mine >= 0)
                bulk_copy(my_ring + slot * C::kTileBytes + lane * kBlock,
                          head_base + (size_t)mine * page_bytes, kBlock, my_bar + 8 * slot);
            return ok;
        };
        uint32_t ok_ring = 0;  // four bits a stage
        const int ahead = min(S, n_tiles);
        {
            uint32_t slot = cons.idx;
            for (int k = 0; k < ahead; ++k) {
                ok_ring = (ok_ring & ~(15u << (4 * slot))) | fetch(k, slot) << (4 * slot);
                if (++slot == S) slot = 0;
            }
        }

        // the query rows as B operands: lane (g, t) holds dimensions 32G + 8t.. of row g
        uint32_t q[NT][NG][4];
        float bias[NT == 1 ? NG : 1][4];  // what a group's scores start from
        bool bad = false;
        const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int G4 = 0; G4 < NG; ++G4) {
                const uint4 v = bf16x8_to_f16x8_sat(q_raw[n][G4], bad);
                q[n][G4][0] = v.x ^ flip;
                q[n][G4][1] = v.y ^ flip;
                q[n][G4][2] = v.z ^ flip;
                q[n][G4][3] = v.w ^ flip;
                if (NT == 1) {
                    float s = 0.0f;
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) {
                        const float2 f = __half22float2(as_h2(q[n][G4][i4]));
                        s += f.x + f.y;
                    }
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
                    bias[NT == 1 ? G4 : 0][0] = -72.0f * __shfl_sync(0xffffffffu, s, 8 * t);
                    bias[NT == 1 ? G4 : 0][1] = -72.0f * __shfl_sync(0xffffffffu, s, 8 * t + 4);
                    bias[NT == 1 ? G4 : 0][2] = bias[NT == 1 ? G4 : 0][0];
                    bias[NT == 1 ? G4 : 0][3] = bias[NT == 1 ? G4 : 0][1];
                }
            }
        if (__any_sync(0xffffffffu, bad) && lane == 0) kv_report(a.err, MOE_KV4_DEVERR_RANGE);

        // tokens that every row sees: below `open`, and from `shut` on
        const int i_lo = div_group(row0, a.gdiv), i_hi = div_group(row0 + rows - 1, a.gdiv);
        const int open = min(rq.end, a.tree ? rq.first : rq.first + i_lo + 1);
        const int shut = a.window > 0 ? rq.first + i_hi - a.window + 1 : 0;

        // m: what a row's probabilities are relative to (see KvAttnArgs); lim: the score from
        // which it moves
        float m[NT][2], lim[NT][2], l[NT][2], acc[NG][2][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = lim[n][0] = lim[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }
#pragma unroll
        for (int x = 0; x < NG * 2 * NT * 4; ++x) (&acc[0][0][0][0])[x] = 0.0f;

        int k = 0;
        for (; k < n_tiles; ++k) {
            const uint32_t slot = cons.idx;
            if (__any_sync(0xffffffffu, !mbar_wait(my_bar + 8 * slot, cons.ph, &abort_flag, a.err))) {
                aborted = true;
                break;
            }
            const uint32_t sb = my_ring + slot * C::kTileBytes;
            const uint32_t ok = (ok_ring >> (4 * slot)) & 15u;
            const int j0 = (tile_lo + k) * kTile;
            const bool full = ok == 15u && j0 + kTile <= open && j0 >= shut;
            // a run of 16 tokens: its block and its first row there
            auto place = [&](int s, uint32_t &base, uint32_t &row) {
                base = sb + (uint32_t)(16 * s / ps) * kBlock;
                row = 16 * s % ps;
            };

            float x[4][NT][4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t base, row;
                place(s, base, row);
                const uint32_t kr = base + (row + tau) * RB + t * (NG * 4);
                const uint32_t sc = base + ps * D + (row + tau) * (NG * 2);
                uint32_t wa[NG], wb[NG], za[NG / 2], zb[NG / 2];
                lds_words(kr, wa);
                lds_words(kr + 8 * RB, wb);
                lds_words(sc, za);
                lds_words(sc + 8 * NG * 2, zb);
                if (NT == 1) {
#pragma unroll
                    for (int G4 = 0; G4 < NG; ++G4) {
                        uint32_t ca[4], cb[4];
                        codes64(wa[G4], a.k, ca);
                        codes64(wb[G4], a.k, cb);
                        float c[4];
                        mma16816(c, ca[0], cb[0], ca[1], cb[1], q[0][G4][0], q[0][G4][1],
                                 bias[NT == 1 ? G4 : 0]);
                        mma16816(c, ca[2], cb[2], ca[3], cb[3], q[0][G4][2], q[0][G4][3]);
                        const float2 fa = __half22float2(as_h2(za[G4 / 2]));
                        const float2 fb = __half22float2(as_h2(zb[G4 / 2]));
                        const float ya = G4 & 1 ? fa.y : fa.x, yb = G4 & 1 ? fb.y : fb.x;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float y = i < 2 ? ya : yb;
                            x[s][0][i] = G4 ? fmaf(c[i], y, x[s][0][i]) : c[i] * y;
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[s][n][i] = 0.0f;
#pragma unroll
                    for (int G4 = 0; G4 < NG; ++G4) {
                        const uint32_t ya = __byte_perm(za[G4 / 2], 0, G4 & 1 ? 0x3232 : 0x1010);
                        const uint32_t yb = __byte_perm(zb[G4 / 2], 0, G4 & 1 ? 0x3232 : 0x1010);
                        uint32_t ca[4], cb[4];
                        codes_scaled(wa[G4], wa[G4] >> 8, a.k, ya, ca);
                        codes_scaled(wb[G4], wb[G4] >> 8, a.k, yb, cb);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816(x[s][n], ca[0], cb[0], ca[1], cb[1], q[n][G4][0], q[n][G4][1]);
                            mma16816(x[s][n], ca[2], cb[2], ca[3], cb[3], q[n][G4][2], q[n][G4][3]);
                        }
                    }
                }
            }
            if (!full) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 8 * n + 2 * t + e, i = div_group(row0 + r, a.gdiv), p = rq.first + i;
                        const int hi = r < rows ? min(p, rq.end - 1) : -1;
                        const int lo = a.window > 0 ? p - a.window : -1;
                        uint64_t word = 0;
                        if (a.tree && r < rows) word = a.tree[rq.q0 + i];
#pragma unroll
                        for (int s = 0; s < 4; ++s)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const int j = j0 + 16 * s + 8 * f + tau;
                                bool see = j <= hi && j > lo && ((ok >> s) & 1u);
                                if (a.tree && j >= rq.first)
                                    see = see && j - rq.first < 64 && ((word >> (j - rq.first)) & 1u);
                                if (!see) x[s][n][2 * f + e] = -INFINITY;
                            }
                    }
            }
            // Maximum and sum of each row (a column here: over the lanes g).  The maximum
            // moves only when some score exceeds it by more than 2^8: the probabilities,
            // relative to m, 2^7 below it, then stay below 2^15, inside fp16, and neither the
            // exchange between the lanes nor the rescaling is paid for every tile.
            uint32_t pb[4][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(x[0][n][e], x[0][n][2 + e]);
#pragma unroll
                    for (int s = 1; s < 4; ++s) v = max3(v, x[s][n][e], x[s][n][2 + e]);
                    top[e] = v;
                }
                if (__any_sync(0xffffffffu, top[0] > lim[n][0] || top[1] > lim[n][1])) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = top[e];
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        const bool up = v > lim[n][e], far = fabsf(v) > a.far;
                        const float base = up ? (far ? v : v - a.raise) : m[n][e];
                        const float r = up ? kv_ex2((m[n][e] - base) * sl2) : 1.0f;
                        if (up) lim[n][e] = far ? v : v + a.lag;
                        m[n][e] = base;
                        l[n][e] *= r;
#pragma unroll
                        for (int G4 = 0; G4 < NG; ++G4)
#pragma unroll
                            for (int c = 0; c < 2; ++c) acc[G4][c][n][e] *= r, acc[G4][c][n][2 + e] *= r;
                    }
                }
                float o0 = m[n][0] == -INFINITY ? 0.0f : -m[n][0] * sl2;
                float o1 = m[n][1] == -INFINITY ? 0.0f : -m[n][1] * sl2;
                if (fmaxf(fabsf(m[n][0]), fabsf(m[n][1])) > a.far) {
                    // the rounding of m * sl2 would be a power of two of its own: such rows
                    // subtract before the scale, and their maximum does not lag
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool far = fabsf(m[n][e]) > a.far && m[n][e] > -INFINITY;
                        const float base = far ? m[n][e] : 0.0f;
                        if (far) (e ? o1 : o0) = 0.0f;
#pragma unroll
                        for (int s = 0; s < 4; ++s) x[s][n][e] -= base, x[s][n][2 + e] -= base;
                    }
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = kv_ex2(fmaf(x[s][n][i], sl2, i & 1 ? o1 : o0));
                    l[n][0] += p[0] + p[2];
                    l[n][1] += p[1] + p[3];
                    pb[s][n][0] = transpose8x8(as_u32(__floats2half2_rn(p[0], p[1])));
                    pb[s][n][1] = transpose8x8(as_u32(__floats2half2_rn(p[2], p[3])));
                }
            }
            // O^T += V^T P^T: lane (g, t) loads tokens t, 4 + (t ^ 1) and eight on
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t base, row;
                place(s, base, row);
                const uint32_t vr = base + ps * RB + row * RB + g * (NG * 2);
                const uint32_t sc = base + ps * D + ps * (NG * 2) + row * (NG * 2);
                const int tok[4] = {t, 4 + (t ^ 1), 8 + t, 12 + (t ^ 1)};
                uint32_t vw[4][NG / 2], z[4][NG / 2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lds_words(vr + tok[i] * RB, vw[i]);
                    lds_words(sc + tok[i] * (NG * 2), z[i]);
                }
                if (!full) {
                    // slots past the sequence (or without a page) hold anything
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j0 + 16 * s + tok[i] >= rq.end || !((ok >> s) & 1u)) {
#pragma unroll
                            for (int c = 0; c < NG / 2; ++c) z[i][c] = 0;
                        }
                }
#pragma unroll
                for (int G4 = 0; G4 < NG; ++G4) {
                    const uint32_t sel = G4 & 1 ? 0x7632 : 0x5410;
                    const uint32_t s0 = __byte_perm(z[0][G4 / 2], z[1][G4 / 2], sel);
                    const uint32_t s1 = __byte_perm(z[2][G4 / 2], z[3][G4 / 2], sel);
                    uint32_t va[4], vb[4];
                    // the same with the bytes of each half exchanged: its high nibbles
                    const uint32_t hsel = G4 & 1 ? 0x6723 : 0x4501;
                    codes_scaled(__byte_perm(vw[0][G4 / 2], vw[1][G4 / 2], sel),
                                 __byte_perm(vw[0][G4 / 2], vw[1][G4 / 2], hsel), a.k, s0, va);
                    codes_scaled(__byte_perm(vw[2][G4 / 2], vw[3][G4 / 2], sel),
                                 __byte_perm(vw[2][G4 / 2], vw[3][G4 / 2], hsel), a.k, s1, vb);
#pragma unroll
                    for (int v = 0; v < 2; ++v)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(acc[G4][v][n], va[2 * v], va[2 * v + 1], vb[2 * v], vb[2 * v + 1],
                                     pb[s][n][0], pb[s][n][1]);
                }
            }
            __syncwarp();
            if (k + S < n_tiles)
                ok_ring = (ok_ring & ~(15u << (4 * slot))) | fetch(k + S, slot) << (4 * slot);
            cons.next();
        }

        if (aborted) {
            // the copies in flight land before the ring is used otherwise or the CTA ends
            // (waits that the abort does not cut short, limited as any other)
            volatile int none = 0;
            Ring left = cons;
            for (int i = k; i < min(n_tiles, k + S); ++i, left.next())
                mbar_wait(my_bar + 8 * left.idx, left.ph, &none, a.err);
            __syncwarp();
        }

        // the segment's result
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
            }
        const bool whole = u == i_u0 && seg_end == i_u1;
        u = seg_end;
        const bool last_seg = u >= u_end;
        if (whole) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * n + 2 * t + e;
                    if (r >= rows) continue;
                    const int i = div_group(row0 + r, a.gdiv), hh = (row0 + r) - i * G;
                    const size_t o = (size_t)(rq.q0 + i) * a.q_heads + h * G + hh;
                    const float inv = l[n][e] > 0.0f ? 1.0f / l[n][e] : 0.0f;
#pragma unroll
                    for (int G4 = 0; G4 < NG; ++G4) {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[G4][0][n][e] * inv,
                                                                        acc[G4][0][n][2 + e] * inv);
                        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[G4][1][n][e] * inv,
                                                                        acc[G4][1][n][2 + e] * inv);
                        *reinterpret_cast<uint2 *>(a.out + o * D + 32 * G4 + 4 * g) =
                            make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                       *reinterpret_cast<const uint32_t *>(&hi));
                    }
                    if (a.lse && g == 0)
                        a.lse[o] = l[n][e] > 0.0f
                                       ? (m[n][e] * sl2 + log2f(l[n][e])) * 0.6931471805599453f
                                       : -INFINITY;
                }
        } else {
            // the last segment's ring is idle and takes the partial; an earlier one's
            // goes to the workspace
            __syncwarp();
            float *slot = last_seg ? reinterpret_cast<float *>(ring + w * C::kRing) : warp_slot;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float *p = slot + (8 * n + 2 * t + e) * C::kPitch;
#pragma unroll
                    for (int G4 = 0; G4 < NG; ++G4)
                        *reinterpret_cast<float4 *>(p + 32 * G4 + 4 * g) =
                            make_float4(acc[G4][0][n][e], acc[G4][0][n][2 + e], acc[G4][1][n][e],
                                        acc[G4][1][n][2 + e]);
                    if (g == 0) p[D] = m[n][e], p[D + 1] = l[n][e];
                }
            if (lane == 0) meta[2 * w + (last_seg ? 1 : 0)] = Meta{i_u0, i_u1, rq.q0, rows, h, row0};
        }
    }
    __syncthreads();

    // The partials in list order; those of one item are a run of neighbouring warps,
    // all in their rings but the run's last, which may be the first of its warp.
    if (w == 0) {
        const Meta me = lane < 2 * W ? meta[lane] : Meta{0, 0, 0, 0, 0, 0};
        const bool has = me.u0 != me.u1;
        const unsigned who = __ballot_sync(0xffffffffu, has);
        const unsigned below = who & ((1u << lane) - 1u);
        const int prev = below ? 31 - __clz(below) : 0;
        const uint32_t prev_u0 = __shfl_sync(0xffffffffu, me.u0, prev);
        const unsigned firsts = __ballot_sync(0xffffffffu, has && (!below || prev_u0 != me.u0));
        if ((firsts >> lane) & 1u) run_of[__popc(firsts & ((1u << lane) - 1u))] = lane;
        if (lane == 0) {
            n_runs = __popc(firsts);
            run_of[__popc(firsts)] = 32 - __clz(who);
        }
    }
    __syncthreads();
    // four dimensions of a row, all parts of its item added up
    auto finish = [&](const Meta &me, int row, int d4, float mm, float ll, float4 s) {
        if (row >= me.rows) return;
        const int rr = me.row0 + row, i = div_group(rr, a.gdiv), hh = rr - i * G;
        const size_t o = (size_t)(me.q0 + i) * a.q_heads + me.h * G + hh;
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x * inv, s.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(s.z * inv, s.w * inv);
        *reinterpret_cast<uint2 *>(a.out + o * D + 4 * d4) = make_uint2(
            *reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        if (a.lse && d4 == 0)
            a.lse[o] = ll > 0.0f ? (mm * sl2 + log2f(ll)) * 0.6931471805599453f : -INFINITY;
    };
    const int runs = n_runs;
    // a warp's share: two rows (D = 64: four) of one item at a time
    constexpr int kGroup = 2 * (32 / (D / 4)), kGroups = C::kRows / kGroup;
    for (int e = w; e < runs * kGroups; e += W) {
        const int run = e / kGroups, from = run_of[run];
        const Meta me = meta[from];
        const int w0 = from >> 1;
        // the run's last slot: the next run's predecessor that is in use
        int to = run_of[run + 1] - 1;
        while (meta[to].u0 != me.u0) --to;
        const int n = (to >> 1) - w0 + 1;
        const float *tail = to & 1 ? nullptr : a.warp_slots + ((size_t)blockIdx.x * W + (to >> 1)) * C::kSlot;
        float *own = me.u0 >= c_lo && me.u1 <= c_hi
                         ? nullptr
                         // the CTA's first item, or its last
                         : a.cta_slots + ((size_t)2 * blockIdx.x + (me.u0 > c_lo ? 1 : 0)) * C::kSlot;
        add_parts<D, 2, 6>(
            n, (e % kGroups) * kGroup, sl2,
            [&](int i) {
                return i == n - 1 && tail ? tail
                                          : reinterpret_cast<const float *>(ring + (w0 + i) * C::kRing);
            },
            [&](int row, int d4, float mm, float ll, float4 s) {
                if (!own) return finish(me, row, d4, mm, ll, s);
                float *p = own + row * C::kPitch;
                *reinterpret_cast<float4 *>(p + 4 * d4) = s;
                if (d4 == 0) *reinterpret_cast<float2 *>(p + D) = make_float2(mm, ll);
            });
    }
    __threadfence();
    __syncthreads();
    // at most two of the runs (the first and the last) are shared with other CTAs
    if (tid < 2) {
        bool last = false;
        const int run = tid == 0 ? 0 : runs - 1;
        if (runs > tid) {
            const Meta me = meta[run_of[run]];
            if (!(me.u0 >= c_lo && me.u1 <= c_hi)) {
                const uint32_t c0 = me.u0 / per, c1 = (me.u1 - 1) / per;  // CTAs of its tiles
                last = atomicAdd(a.counters + c0, 1) == (int)(c1 - c0);
                if (last) a.counters[c0] = 0;
            }
        }
        last_of[tid] = last;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (!last_of[k]) continue;
        const Meta me = meta[run_of[k == 0 ? 0 : runs - 1]];
        const uint32_t c0 = me.u0 / per, c1 = (me.u1 - 1) / per;
        __threadfence();
        const int odd = me.u0 > c0 * per ? 1 : 0;  // in its first CTA the item is the last one
        constexpr int kStep = 32 / (D / 4);
        for (int row = w * kStep; row < C::kRows; row += W * kStep)
            add_parts<D, 1, 12>(
                (int)(c1 - c0) + 1, row, sl2,
                [&](int i) { return a.cta_slots + ((size_t)2 * (c0 + i) + (i ? 0 : odd)) * C::kSlot; },
                [&](int r, int d4, float mm, float ll, float4 s) { finish(me, r, d4, mm, ll, s); });
    }
    if (a.beside) pdl_wait();
}

template <int D, int NT, int PS>
cudaError_t launch(const KvAttnArgs &a, int grid, cudaStream_t s) {
    using C = Cfg<D, NT>;
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(kv4_decode_kernel<D, NT, PS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) set[dev] = true;
    }
    auto c = pdl_config((unsigned)grid, C::kWarps * 32, C::kSmem, s);
    cudaLaunchAttribute at{};
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return cudaLaunchKernelEx(&c, kv4_decode_kernel<D, NT, PS>, a);
}

template <int D, int NT>
cudaError_t launch_ps(const KvAttnArgs &a, int grid, cudaStream_t s) {
    switch (a.pool.ps) {
        case 16: return launch<D, NT, 16>(a, grid, s);
        case 32: return launch<D, NT, 32>(a, grid, s);
        default: return launch<D, NT, 64>(a, grid, s);
    }
}

}  // namespace

size_t kv4_decode_slot_bytes(int D, int ctas) {
    // NT = 2 has the larger slots, NT = 1 the more warps
    const size_t one = (size_t)8 * (D + 4) * 4;
    return (size_t)ctas * (2 * 2 * one + (size_t)16 * one);
}

cudaError_t launch_kv4_decode(KvAttnArgs a, int D, int max_rows, void *slots, int ctas,
                              cudaStream_t s) {
    const int nt = max_rows <= 8 ? 1 : 2;
    const size_t slot = (size_t)8 * nt * (D + 4);
    a.cta_slots = reinterpret_cast<float *>(slots);
    a.warp_slots = a.cta_slots + 2 * slot * ctas;
    a.min_units = 4;  // a tile for each quarter of an SM: short calls spread over the GPU
    // no more CTAs than the largest possible list of units fills
    const long long tiles = (long long)(a.max_kv + kTile - 1) / kTile + 1;
    const long long row_tiles = ((long long)max_rows + 8 * nt - 1) / (8 * nt);
    long long most = tiles * row_tiles * a.pool.hkv * a.batch.requests;
    most = (most + a.min_units - 1) / a.min_units;
    const int grid = (int)(most < 1 ? 1 : most < ctas ? most : ctas);
    if (D == 128) return nt == 1 ? launch_ps<128, 1>(a, grid, s) : launch_ps<128, 2>(a, grid, s);
    return nt == 1 ? launch_ps<64, 1>(a, grid, s) : launch_ps<64, 2>(a, grid, s);
}

}  // namespace moe
