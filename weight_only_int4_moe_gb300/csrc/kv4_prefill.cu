// Attention over the 4-bit cache for many query rows (include/moe_kv4.h): prompts,
// chunks and larger verify batches, where the products are the bound.
//
// An item is up to 256 query rows that share a kv head (its group's heads of
// consecutive tokens), two tiles of 128 for tcgen05.mma, against tiles of 128
// tokens.  Per tile of tokens and rows,
//   S = Q K^T   (128 x 128 x D, both operands fp16 in shared memory)
//   P = 2^(S - m) in fp16, written over S in tensor memory
//   O += P V    (128 x D x 128, P from tensor memory, V from shared memory)
// with m, 2^7 below the row's running maximum, and the sum of a row in the two threads
// that own the row.  O is rescaled only when a row's maximum has grown by more than 2^8
// since its last rescale, a method known from published attention kernels (P then stays
// below 2^15, inside fp16, and the quotient O / l does not depend on m).
//
// Roles of the 28 warps: two pairs of warpgroups each own one tile of rows, a thread
// half of a row's columns (they load its Q, do the softmax, write the output; the
// maximum of a row passes between its two threads through shared memory); one
// warpgroup turns K's codes into fp16 operand tiles and one V's, their loads one tile
// ahead in registers; a warp for each tile of rows issues its MMAs, so that the softmax
// of one runs under the products of the other; one more warp finds the CTA's runs of
// work.  An item of up to 128 rows has one tile of rows: both pairs of warpgroups take
// it, each every other tile of tokens, and the first adds up their two results.
//
// The scores are worked on in half tiles of 64 tokens, two buffers a tile of rows: the
// products of one half run under the softmax of the other (605 -> 513 us below against
// whole tiles, although an MMA of 64 columns with both operands in shared memory takes
// 48 cycles where 32 would do: its operands' bytes bound it).  A row in two threads: with
// a thread a whole row, half the warps and twice the registers each, a tile's softmax
// took about 1900 cycles, most of it latency.
// K tiles are K-major, V tiles are left in token order and read N-major; the order of
// V's columns is the order in which its codes unpack, undone when the output is
// written.
//
// The list of (request, row tile, kv head) items' token tiles is cut into equal
// runs, one a CTA; parts of an item are joined through the workspace by the last
// CTA to arrive, in list order.
//
// Measured: 4096 new tokens behind 4096 cached ones, 32 heads over 8 kv heads of 128:
// 428 us, 962 TFLOP/s of the 1901 that a large bf16 product reaches; 10 verify streams of
// up to 5000 tokens, up to 63 rows each: 50 us.  A tile of 256 rows and 128 tokens takes about
// 4900 cycles, its MMAs alone 2520.  With the softmax's arithmetic, or the unpacking,
// taken out the first, then at 447 us, fell to 414 and to 383, without either to 350: what
// remains is the round trip between the products and the softmax.  A whole tile's more
// scores in flight would need tensor memory that is all in use (O 256 columns, S 256).
// The verify streams' items are bound by the two warpgroups that unpack, about 4000 cycles
// a tile; their loads go through registers one tile ahead.
#include <atomic>

#include "dequant.cuh"
#include "kv4_launch.cuh"

namespace moe {

namespace {

// What a row is relative to before any score: finite, so that differences are numbers.
constexpr float kLow = -3e38f;
constexpr int kTok = 128;        // tokens of a unit
// Units before an item's first tile that hold no work: what a new item costs (its
// queries, filling the pipeline, its output) in tiles.  Without them a CTA whose run
// is many short items ends long after the others (a verify batch of ragged lengths:
// 119 us against a median of 42 us).
constexpr int kPad = 4;
constexpr int kRowsItem = 256;
constexpr int kChunks = 1024;
constexpr uint32_t kRuns = 8;    // of the CTA's list, in shared memory at a time
constexpr int kThreads = 896;
constexpr uint32_t kTmemCols = 512;
// Registers a thread of each role (multiples of 8).  The seven warpgroups' shares add
// up to what the block is launched with, 7 x 72.
constexpr int kRegsLaunch = 72, kRegsSoftmax = 80, kRegsCodes = 64, kRegsMma = 56;
static_assert(4 * kRegsSoftmax + 2 * kRegsCodes + kRegsMma == 7 * kRegsLaunch, "register shares");
static_assert(kThreads * kRegsLaunch <= 65536, "the register file");
// Before the block's common end every warp returns to kRegsLaunch.  Those that take
// registers back wait at this barrier until those that give them up have done so,
// and until the softmax warps have had theirs: a warp with no work that took its
// share back early would keep it from a softmax warp that still waits for it.
constexpr uint32_t kBarRegs = 1, kBarBoth = 2;  // kBarBoth: both row tiles' threads
constexpr uint32_t kBarPair = 3;                // + 0..7: the two warps that share 32 rows

template <int D>
struct Cfg {
    static constexpr int kTileBytes = kTok * D * 2;   // an operand tile
    static constexpr int kQ = 0;                      // two tiles of rows
    static constexpr int kK = 2 * kTileBytes;         // two K tiles, two V tiles
    static constexpr int kV = 4 * kTileBytes;
    static constexpr int kSmem = 6 * kTileBytes + 1024;
    static constexpr int kPitch = D + 4;
    static constexpr int kSlot = kRowsItem * kPitch;
    static constexpr int kLoads = D == 128 ? 4 : 2;   // 16-byte loads a thread for K (and V)
};

// S and P: by row tile and half tile (2 m + sub); kPv: by row tile, after every P V.
// A wait names a phase by its parity, so it is only sound while the barrier is at most
// one lap away from the phase waited for.  The rings of two (K, V) and Q hold that for a
// MMA warp because
//  - within a run it waits for its own tiles in order, and a tile that it has to consume
//    cannot be overwritten, so no ring runs ahead of it;
//  - in a narrow run it skips the other warp's tiles.  K and Q: the next run's kQFull
//    follows kQEmpty, so all scores of the old run, and with them all its K, are done.
//    V: the old run's last tile may still be on its way to the slot of this warp's first
//    tile of the new run, whose wait would pass a lap early and multiply stale values.  The
//    first tile's P comes after kBarBoth of the old run, so after its last product with
//    V: a run's first kVFull is waited for behind that P.
enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kQFull = 8, kPv = 10, kSFull = 12, kPFull = 16, kQEmpty = 20, kOFull = 22, kRunFull = 24, kRunEmpty = 32, kDrain = 40, kBars = 42 };

struct Request {
    int q0, m, first, end, rows, row_tiles;
};

MOE_DEV Request request_of(const KvAttnArgs &a, int b) {
    Request r;
    r.q0 = a.batch.cu_q[b];
    const int q1 = a.batch.cu_q[b + 1];
    r.m = q1 - r.q0;
    const int len = a.batch.kv_len[b];
    r.first = len - r.m;
    r.end = (int)min((long long)min(len, kKvMaxLen), (long long)a.batch.stride * a.pool.ps);
    r.rows = r.m * a.group;
    // (a row range outside the batch's tokens is no request; compared before r.m is used,
    // as the difference of two ints may wrap)
    const bool mine = r.q0 >= 0 && q1 > r.q0 && q1 <= a.batch.tokens && r.rows >= a.rows_lo &&
                      r.rows <= a.rows_hi;
    r.row_tiles = mine ? (r.rows + kRowsItem - 1) / kRowsItem : 0;
    return r;
}

// Token tiles of a row tile: [lo, lo + n).
MOE_DEV int tiles_of(const KvAttnArgs &a, const Request &r, int rt, int &lo) {
    const int i_lo = div_group(rt * kRowsItem, a.gdiv);
    const int i_hi = div_group(min(r.rows, (rt + 1) * kRowsItem) - 1, a.gdiv);
    const int hi = max(0, min(r.end, r.first + i_hi + 1));
    lo = (a.window > 0 ? max(0, r.first + i_lo - a.window + 1) : 0) / kTok;
    return max(1, (hi + kTok - 1) / kTok - lo);
}

// Units of a request, by a whole warp.
MOE_DEV uint32_t request_units(const KvAttnArgs &a, const Request &r) {
    uint32_t n = 0;
    int lo;
    for (int rt = threadIdx.x & 31; rt < r.row_tiles; rt += 32) n += tiles_of(a, r, rt, lo) + kPad;
    return __reduce_add_sync(0xffffffffu, n) * a.pool.hkv;
}

// A run of one item's tiles that a CTA works on.
struct Segment {
    Request r;
    int b, rt, h, tile0, n;       // tile0: the first token tile of the run
    uint32_t i_u0, i_u1;          // the item's tiles as units
    int rows;                     // of the item
    bool whole;
};

struct Shared {
    uint64_t bar[kBars];
    uint32_t tmem, warp_tot[kThreads / 32];
    int abort_flag, last_of[2];
    // The CTA's runs, a few ahead: one warp finds them, the others read them here.  stop:
    // the number of the run at which the list breaks off (a wait gave up).
    Segment run[kRuns];
    volatile uint32_t stop;
    uint32_t ok[8];              // runs of 16 tokens that have a page, by tile
    uint32_t prefix[kChunks + 1];
    int4 see[2][2][128];         // by row tile, half and row: lo, hi, first new token
    uint64_t word[2][2][128];    // and the row's word of the tree
    float top[2][2][2][128];     // a tile's row maxima: by parity, row tile, half
    uint32_t part_u0[2], part_u1[2];
    int part_q0[2], part_h[2], part_row0[2], part_rows[2];
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
        while (u < u_end) {
            s.r = request_of(a, b);
            while (true) {
                const uint32_t n = per_chunk == 1 ? prefix[b + 1] - prefix[b] : request_units(a, s.r);
                if (u < b_u0 + n) break;
                if (b + 1 >= a.batch.requests) return false;  // the lengths changed under the call
                b_u0 += n;
                s.r = request_of(a, ++b);
            }
            // the row tile: 32 at a time
            const int lane = threadIdx.x & 31, hkv = a.pool.hkv;
            uint32_t at = u - b_u0, base = 0;
            for (int rt0 = 0;; rt0 += 32) {
                int lo = 0;
                const int rt = rt0 + lane;
                const uint32_t n = rt < s.r.row_tiles ? (uint32_t)(tiles_of(a, s.r, rt, lo) + kPad) : 0u;
                uint32_t x = n * hkv;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
                    if (lane >= d) x += y;
                }
                const unsigned who = __ballot_sync(0xffffffffu, at < base + x);
                if (!who) {
                    if (rt0 >= s.r.row_tiles) return false;
                    base += __shfl_sync(0xffffffffu, x, 31);
                    continue;
                }
                const int l = __ffs(who) - 1;
                s.rt = rt0 + l;
                const uint32_t span = __shfl_sync(0xffffffffu, n, l);
                const uint32_t rt_u0 = base + __shfl_sync(0xffffffffu, x, l) - span * hkv;
                s.h = (int)((at - rt_u0) / span);
                s.i_u0 = b_u0 + rt_u0 + s.h * span + kPad;  // its tiles
                s.i_u1 = s.i_u0 - kPad + span;
                s.tile0 = __shfl_sync(0xffffffffu, lo, l);
                break;
            }
            u = max(u, s.i_u0);
            if (u >= u_end) return false;
            s.tile0 += (int)(u - s.i_u0);
            s.b = b;
            const uint32_t end = min(u_end, s.i_u1);
            s.n = (int)(end - u);
            s.whole = u == s.i_u0 && end == s.i_u1;
            s.rows = min(kRowsItem, s.r.rows - s.rt * kRowsItem);
            u = end;
            return true;
        }
        return false;
    }
};

// Run number idx of the CTA's list, or null at its end.  The warp that writes the list
// either publishes a run or stops at it, within the limit of its own waits, so that all
// warps see the same list.  (The limit here only guards that: 2^22 polls of up to 20 us.)
MOE_DEV const Segment *run_at(Shared &sh, uint32_t idx) {
    const uint32_t bar = smem_u32(&sh.bar[kRunFull + idx % kRuns]), ph = (idx / kRuns) & 1u;
    for (uint32_t it = 0; it < (1u << 22); ++it) {
        if (__any_sync(0xffffffffu, mbar_try_wait(bar, ph))) {
            const Segment *r = &sh.run[idx % kRuns];
            return r->n ? r : nullptr;
        }
        if (__any_sync(0xffffffffu, sh.stop == idx)) return nullptr;
    }
    return nullptr;
}
// A warp needs run idx no more.
MOE_DEV void run_done(Shared &sh, uint32_t idx) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sh.bar[kRunEmpty + idx % kRuns]));
}
// The warp that finds the runs.
MOE_DEV void write_runs(const KvAttnArgs &a, Shared &sh, Walk walk) {
    for (uint32_t idx = 0;; ++idx) {
        Segment sg;
        const bool more = walk.next(a, sg);
        if (!more) sg.n = 0;
        if (idx >= kRuns &&
            __any_sync(0xffffffffu, !mbar_wait(smem_u32(&sh.bar[kRunEmpty + idx % kRuns]),
                                               (idx / kRuns - 1) & 1u, &sh.abort_flag, a.err, 200))) {
            if ((threadIdx.x & 31) == 0) sh.stop = idx;
            return;
        }
        if ((threadIdx.x & 31) == 0) {
            sh.run[idx % kRuns] = sg;
            mbar_arrive(smem_u32(&sh.bar[kRunFull + idx % kRuns]));
        }
        __syncwarp();
        if (!more) return;
    }
}

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

// S = Q K^T for half a tile of tokens: D / 16 MMAs, operands in column blocks of 64
// dimensions.
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

// O (+)= P V for half a tile: four MMAs of 16 tokens each; P's columns are 0..15 for
// the first 32 tokens and 32..47 for the others.
MOE_DEV void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 32;\n\tadd.u32 a3, %1, 40;\n\t"
        "add.u64 b1, %2, 128;\n\tadd.u64 b2, %2, 256;\n\tadd.u64 b3, %2, 384;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
        "r"(p_tmem), "l"(desc_n_major(v)), "r"(idesc), "r"(accumulate)
        : "memory");
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
// Waits for the thread's loads; the registers pass through, so that no use of them can
// come before the wait.
MOE_DEV void tmem_wait_ld(uint32_t *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : KV4_P8(v, 0), KV4_P8(v, 8), KV4_P8(v, 16), KV4_P8(v, 24)::"memory");
}

// One instruction of the ALU pipe, which has half the lanes of the FMA pipe.
MOE_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Which of the tokens j0..j0+31 a row sees, as bits: lo < j <= hi, in a run of 16
// that has a page, and by the row's word for the new tokens (from `first` on).
MOE_DEV uint32_t visible32(int j0, int lo, int hi, uint32_t ok, bool tree, uint64_t word, int first) {
    const int b = hi - j0, a = lo + 1 - j0;
    uint32_t see = b < 0 ? 0u : b >= 31 ? 0xffffffffu : (2u << b) - 1u;
    see &= a <= 0 ? 0xffffffffu : a >= 32 ? 0u : 0xffffffffu << a;
    see &= (ok & 1u ? 0xffffu : 0u) | (ok & 2u ? 0xffff0000u : 0u);
    if (tree) {
        const int d = j0 - first;  // index of j0 among the new tokens
        if (d >= 0)
            see &= d < 64 ? (uint32_t)(word >> d) : 0u;
        else if (d > -32)
            see &= (uint32_t)(word << -d) | ((1u << -d) - 1u);
    }
    return see;
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

// A word's four nibble pairs as (q - 8) * s in fp16, exact: (16 + q) * s - 24 * s.
MOE_DEV void scaled_codes(uint32_t w, const KvConsts &k, uint32_t s, uint32_t (&x)[4]) {
    const __half2 m24 = __hmul2(as_h2(s), as_h2(k.cm24));
    const uint32_t v = w >> 8;
    const uint32_t t[4] = {w * k.c64, w * k.c4, v * k.c64, v * k.c4};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = as_u32(__hfma2(as_h2((t[i] & k.nib6) | k.magic16), as_h2(s), m24));
}

MOE_DEV void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Multiplies the thread's half row of O (rarely needed: see the file's head).
template <int D>
MOE_DEV void scale_o(uint32_t o_at, float f) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        float o[16];
        tmem_ld_32x32b_x16_wait(o_at + 16 * c, o);
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[e] * f);
        tmem_st16(o_at + 16 * c, v);
    }
}

// A thread's part of one tile of codes and scales, on its way from global memory,
// and which of its rows hold a token.
template <int D>
struct Packed {
    uint4 c[Cfg<D>::kLoads];
    uint32_t z[Cfg<D>::kLoads][D / 64];
    uint32_t live;
};

// The row that a thread unpacks first.  The eight lanes of a store phase hold two
// rows (D = 64: four); their order puts the swizzled 16-byte chunks that the lanes
// store at once into different banks: K stores chunks 4G + t of all t together, so
// rows four apart, V stores every other chunk, so neighbouring rows.
template <int D, int part>
MOE_DEV int row_of_lane(int dt) {
    const int warp = dt >> 5, l = dt & 31;
    if (D == 128) return 8 * warp + (part == 0 ? (l >> 3) + 4 * ((l >> 2) & 1) : l >> 2);
    if (part == 1) return 16 * warp + (l >> 1);
    const int i = (l >> 1) & 3, j = l >> 3;
    return 16 * warp + (i & 1) + 4 * (i >> 1) + 2 * (j & 1) + 8 * (j >> 1);
}

// The warpgroup that turns one side's codes (part 0: K, 1: V) into operand tiles.
template <int D, int part>
MOE_DEV void unpack_role(const KvAttnArgs &a, Shared &sh, uint32_t smem) {
    using C = Cfg<D>;
    constexpr int kLanesRow = D == 128 ? 4 : 2;  // 16-byte chunks of a row
    constexpr int kStep = 128 / kLanesRow;       // rows of one load of the group
    const int lane = threadIdx.x & 31, dt = threadIdx.x & 127, ch = dt % kLanesRow;
    const int row_l = row_of_lane<D, part>(dt);
    constexpr int NG = D / 32;
    const int ps = a.pool.ps, ppt = kTok >> (31 - __clz(ps)), hkv = a.pool.hkv;
    const uint32_t full = smem_u32(&sh.bar[part ? kVFull : kKFull]);
    const uint32_t empty = smem_u32(&sh.bar[part ? kVEmpty : kKEmpty]);
    // where the thread's first chunk goes (tile_at is the same for rows kStep apart)
    const int first = part == 0 ? (D == 128 ? ch : 2 * ch) : (D == 128 ? 2 * ch : 4 * ch);
    const uint32_t at0 = smem + (part ? C::kV : C::kK) + tile_at(row_l, first);
    // The tile whose loads are requested.  Each of them goes out as soon as the tile
    // before has left its registers.  Kept from the run: the head's blocks (from the
    // thread's chunk on), the tiles left, the tokens left, the table's first,
    // next and last entry.
    const int ps_log = 31 - __clz(ps);
    const uint32_t page_bytes = a.pool.block * hkv;
    const uint8_t *head = nullptr;
    const int32_t *table = nullptr;
    int tiles_left = 0, left = 0, id_at = 0, entry = 0, entries = 0, ids = -1, ids_next = -1, from = 0;
    bool reports = false;
    uint32_t run_idx = 0;
    // page ids: lane l holds the tile's and the following ones, 32 in all, then 32 more
    auto next_ids = [&] {
        ids = ids_next;
        if (entry + lane < from) ids = -1;
        if ((unsigned)ids >= (unsigned)a.pool.n_pages) {
            if (reports && entry + lane >= from && entry + lane < entries)
                kv_report(a.err, MOE_KV4_DEVERR_PAGE);
            ids = -1;
        }
        entry += 32;
        ids_next = entry + lane < entries ? table[entry + lane] : -1;
        id_at = 0;
    };
    uint32_t ok_next = 0;
    auto advance = [&]() -> bool {
        if (tiles_left == 0) {
            const Segment *run = run_at(sh, run_idx);
            if (!run) return false;
            const Segment &sg = *run;
            table = a.batch.tables + (size_t)sg.b * a.batch.stride;
            head = a.pool.base + (size_t)sg.h * a.pool.block;
            reports = part == 0 && sg.h == 0 && dt < 32;
            // (not the pages that the window of the run's first row has left behind: they may
            // be gone, or hold anything)
            from = a.window > 0
                       ? max(0, sg.r.first + div_group(sg.rt * kRowsItem, a.gdiv) - a.window + 1) >> ps_log
                       : 0;
            tiles_left = sg.n;
            left = sg.r.end - sg.tile0 * kTok;
            entry = sg.tile0 * ppt;
            entries = min((sg.tile0 + sg.n) * ppt, (sg.r.end + ps - 1) >> ps_log);
            run_done(sh, run_idx++);
            ids_next = entry + lane < entries ? table[entry + lane] : -1;
            next_ids();
        } else {
            left -= kTok;
            id_at += ppt;
            if (id_at == 32) next_ids();
        }
        --tiles_left;
        if (part == 0) {
            const unsigned have = __ballot_sync(0xffffffffu, ids >= 0) >> id_at;
            ok_next = 0;
            for (int i = 0; i < ppt; ++i)
                if ((have >> i) & 1u) ok_next |= ((1u << (ps / 16)) - 1u) << (i * (ps / 16));
        }
        return true;
    };
    Packed<D> pk;
    // (nothing waits for a load here: rows without a token load page 0 and are zeroed when
    // they are unpacked).  All page ids come first: a warp has six scoreboards, and a
    // shuffle that shared one with a load would wait for the load.
    auto request = [&] {
        int id[C::kLoads];
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i)
            id[i] = __shfl_sync(0xffffffffu, ids, id_at + ((i * kStep + row_l) >> ps_log));
        pk.live = 0;
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
            pk.live |= (id[i] >= 0 && i * kStep + row_l < left ? 1u : 0u) << i;
            id[i] = max(id[i], 0);
            asm volatile("" : "+r"(id[i])::"memory");
        }
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
            const int slot = (i * kStep + row_l) & (ps - 1);
            const uint8_t *blk = head + (size_t)(uint32_t)id[i] * page_bytes;
            pk.c[i] = *reinterpret_cast<const uint4 *>(blk + (part * ps + slot) * (D / 2) + 16 * ch);
            const uint8_t *sc = blk + ps * D + (part * ps + slot) * (NG * 2);
            if constexpr (D == 128) {
                const uint2 v = *reinterpret_cast<const uint2 *>(sc);
                pk.z[i][0] = v.x;
                pk.z[i][1] = v.y;
            } else {
                pk.z[i][0] = *reinterpret_cast<const uint32_t *>(sc);
            }
        }
    };
    Ring ring(2);
    uint32_t tiles = 0;
    bool more = advance();
    if (more) request();
    while (more) {
        const uint32_t ok = ok_next;
        more = advance();
        if (__any_sync(0xffffffffu, !mbar_wait(empty + 8 * ring.idx, ring.ph ^ 1, &sh.abort_flag, a.err)))
            return;
        if (part == 0 && dt == 0) sh.ok[tiles & 7] = ok;
        ++tiles;
        const uint32_t dst = at0 + ring.idx * C::kTileBytes;
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
            const uint32_t words[4] = {pk.c[i].x, pk.c[i].y, pk.c[i].z, pk.c[i].w};
            uint32_t z[D / 64];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) z[c] = (pk.live >> i) & 1u ? pk.z[i][c] : 0u;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // K's word (t, G) holds dimensions 32G + 8t.., the row's chunk 4G + t; V's
                // piece g of groups 2p and 2p + 1 is the column chunk 8p + g.  Seen from the
                // thread's first chunk: a change of chunk bits, which the swizzle keeps, and
                // a column block.
                const int G = D == 128 ? u : u & 1, pp = D == 128 ? u & 1 : 0;
                const uint32_t flip = part == 0 ? (G & 1) * 64u + (D == 128 ? 0u : (u >> 1) * 16u)
                                                : (D == 128 ? (u >> 1) * 16u : u * 16u);
                const uint32_t block = part == 0 ? G >> 1 : pp;
                const uint32_t s = part == 0 ? as_u32(G & 1 ? __high2half2(as_h2(z[G / 2])) : __low2half2(as_h2(z[G / 2]))) : z[pp];
                uint32_t x[4];
                scaled_codes(words[u], a.k, s, x);
                sts128((dst ^ flip) + block * (kTok * 128) + i * (kStep * 128), x[0], x[1], x[2], x[3]);
            }
        }
        fence_proxy_async_shared();
        if (!(kDebugBounds && part == 1 && blockIdx.x == 0 && (int)tiles - 1 == a.skip_tile))
            mbar_arrive(full + 8 * ring.idx);
        request();  // (past the last tile: that one again)
        ring.next();
    }
}

template <int N>
MOE_DEV void more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
MOE_DEV void fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A tile of up to 128 query rows, from row_base of the request on: 16-byte chunks,
// converted to fp16 and swizzled, by 256 threads (id).  (fp16, as both operands of a
// product have one type and K's values are exact there: bf16's eight bits fit from 2^-14
// up, smaller queries keep steps of 2^-24, larger ones than 65504 are reported.)
template <int D>
MOE_DEV void load_q(const KvAttnArgs &a, const Segment &sg, uint32_t dst, int row_base, int n_rows, int id) {
    bool bad = false;
    const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int c0 = 0; c0 < D / 16; c0 += 4) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = id + 256 * (c0 + e), qr = c / (D / 8), ch = c % (D / 8);
            const int i = div_group(row_base + qr, a.gdiv), hh = row_base + qr - i * a.group;
            v[e] = make_uint4(0, 0, 0, 0);
            if (qr < n_rows)
                v[e] = *reinterpret_cast<const uint4 *>(a.q + (size_t)(sg.r.q0 + i) * a.q_stride +
                                                        (size_t)(sg.h * a.group + hh) * D + 8 * ch);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = id + 256 * (c0 + e), qr = c / (D / 8), ch = c % (D / 8);
            const uint4 x = bf16x8_to_f16x8_sat(v[e], bad);
            sts128(dst + tile_at(qr, ch), x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip);
        }
    }
    if (__any_sync(0xffffffffu, bad) && (id & 31) == 0) kv_report(a.err, MOE_KV4_DEVERR_RANGE);
    fence_proxy_async_shared();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const KvAttnArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Shared sh;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, hkv = a.pool.hkv;
    pdl_wait();
    if (a.beside) pdl_launch_dependents();
    if (tid == 0) {
        sh.abort_flag = 0;
        const int counts[21] = {128, 2, 128, 2, 256, 1, 1, 1, 256, 256, 2, 1, 1, 1, 1, 1, 26, 26, 26, 26, 1};
        sh.stop = 0xffffffffu;
        for (int i = 0; i < kBars; ++i) mbar_init(smem_u32(&sh.bar[i]), counts[i / 2]);
        mbar_fence_init();
        sh.part_u0[0] = sh.part_u1[0] = sh.part_u0[1] = sh.part_u1[1] = 0;
    }
    if (w == 27) {
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
                for (int rt = 0; rt < r.row_tiles; ++rt) n += (uint32_t)(tiles_of(a, r, rt, lo) + kPad) * hkv;
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
    const float sl2 = a.sl2;
    auto bar = [&](int i) { return smem_u32(&sh.bar[i]); };
    // S of the row tiles' half tiles, then their O; P lies over the first half of either
    // 32 columns of S
    auto s_col = [&](int m, int sub) { return tmem + 128u * m + 64u * sub; };
    auto o_col = [&](int m) { return tmem + 256u + 128u * m; };
    int *abort_flag = &sh.abort_flag;

    if (c_lo < c_hi) {
        if (w < 16) {
            // ------------------------------------------- softmax of a tile of rows --
            more_regs<kRegsSoftmax>();
            // the thread's row tile, half of the columns and row
            const int m = w >> 3, half = (w >> 2) & 1, r = tid & 127;
            const uint32_t lane_off = (uint32_t)(32 * (w & 3)) << 16;
            const uint32_t s_at = s_col(m, 0) + lane_off + 32u * half;  // P over its first half
            const uint32_t pair_bar = kBarPair + 4 * m + (w & 3);
            const uint32_t o_at = o_col(m) + lane_off + (D / 2) * half;
            // s_ph: phase of S; pv: products with V so far; t0: tiles of earlier runs
            uint32_t s_ph = 0, o_ph = 0, pv = 0, e_ph = 0, t0 = 0;
            bool dead = false;
            // the queries of this warpgroup pair's rows, where it loads any
            auto queries = [&](const Segment &x) {
                load_q<D>(a, x, smem + C::kQ + m * C::kTileBytes, x.rt * kRowsItem + m * 128,
                          min(128, x.rows - m * 128), tid & 255);
                mbar_arrive(bar(kQFull + m));
            };
            uint32_t run_idx = 0;
            const Segment *run = run_at(sh, 0);
            if (run && m * 128 < run->rows) queries(*run);
            while (run) {
                const Segment &sg = *run;
                // up to 128 rows: both pairs take them, every other tile of tokens each
                const bool narrow = sg.rows <= 128;
                const int first = narrow ? m : 0, step = narrow ? 2 : 1;
                const int row_base = sg.rt * kRowsItem + (narrow ? 0 : m * 128);
                const int n_rows = min(128, sg.rows - (narrow ? 0 : m * 128));
                const int i = div_group(row_base + r, a.gdiv), hh = row_base + r - i * a.group;
                const bool live = r < n_rows;
                const int p = sg.r.first + i;
                const int hi = live ? min(p, sg.r.end - 1) : -1;
                const int lo = a.window > 0 ? p - a.window : -1;
                // for the tiles at the edges only: not kept in registers
                sh.see[m][half][r] = make_int4(lo, hi, sg.r.first, 0);
                if (a.tree) sh.word[m][half][r] = live ? a.tree[sg.r.q0 + i] : 0;
                // tokens that every row of the warp sees
                const int open = __reduce_min_sync(0xffffffffu, live ? (a.tree ? min(hi + 1, sg.r.first) : hi + 1)
                                                                     : INT32_MAX);
                const int shut = __reduce_max_sync(0xffffffffu, live ? lo + 1 : 0);
                float top = kLow, sum = 0.0f;
                int j0 = (sg.tile0 + first) * kTok + 32 * half;
                uint32_t at = t0 + first;  // the tile among all of the CTA's
                const int mine = sg.n > first ? (sg.n - first + step - 1) / step : 0;
#pragma unroll 1
                for (int left = 2 * mine; left > 0; --left) {
                    // half a tile: the first of a tile where left is even
                    const uint32_t sub = left & 1, s_sub = s_at + 64u * sub;
                    // a wait that gave up (a kernel bug, reported) leaves the loop's shape
                    // as it is: the tile's other warps count on this one at the barriers
                    if (!dead)
                        dead = __any_sync(0xffffffffu, !mbar_wait(bar(kSFull + 2 * m + sub), s_ph, abort_flag, a.err));
                    tc_fence_after();
                    const uint32_t ok = sh.ok[at & 7] >> (4 * sub + 2 * half);
                    float *swap = &sh.top[sub][m][0][r];
                    uint32_t v[32];
                    tmem_ld32(s_sub, v);
                    tmem_wait_ld(v);
                    if ((ok & 3u) != 3u || j0 + 32 > open || j0 < shut) {
                        const int4 edge = sh.see[m][half][r];
                        const uint32_t see = visible32(j0, edge.x, edge.y, ok, a.tree != nullptr,
                                                       a.tree ? sh.word[m][half][r] : 0, edge.z);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((see >> e) & 1u)) v[e] = 0xff800000u;  // -inf
                    }
                    float mx[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = fmaxf(__uint_as_float(v[e]), __uint_as_float(v[e + 4]));
#pragma unroll
                    for (int e = 8; e < 32; e += 8)
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            mx[f] = max3(mx[f], __uint_as_float(v[e + f]), __uint_as_float(v[e + f + 4]));
                    float now = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                    // the other half's maximum
                    swap[128 * half] = now;
                    named_bar_sync(pair_bar, 64);
                    now = fmaxf(now, swap[128 * (half ^ 1)]);
                    // top: what the row's probabilities are relative to (see KvAttnArgs); it
                    // moves when the maximum has grown by more than 2^8, and with a run's first
                    const bool grow = now - top > a.reach;
                    if (__any_sync(0xffffffffu, grow)) {
                        if (fabsf(now) <= a.far) now -= a.raise;
                        const float f = grow ? kv_ex2((top - now) * sl2) : 1.0f;
                        if (grow) top = now;
                        sum *= f;
                        if (left != 2 * mine) {
                            // O is free once the last product with V is done
                            if (!dead)
                                dead = __any_sync(0xffffffffu, !mbar_wait(bar(kPv + m), (pv - 1) & 1u, abort_flag, a.err));
                            tc_fence_after();
                            scale_o<D>(o_at, f);
                        }
                    }
                    ++pv;
                    // the difference first: the rounding of top * sl2, which one FMA behind the
                    // scale would need, is a power of two of its own for large scores
                    const uint64_t sc2 = pack2(sl2, sl2), top2 = pack2(-top, -top);
                    uint64_t sum2[2] = {pack2(sum, 0.0f), 0};
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float x, y;
                        unpack2(fma2(add2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), top2), sc2, 0), x, y);
                        x = kv_ex2(x);
                        y = kv_ex2(y);
                        sum2[(e >> 1) & 1] = add2(sum2[(e >> 1) & 1], pack2(x, y));
                        p[e / 2] = as_u32(__floats2half2_rn(x, y));
                    }
                    tmem_st16(s_sub, p);
                    {
                        float x, y;
                        unpack2(add2(sum2[0], sum2[1]), x, y);
                        sum = x + y;
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(bar(kPFull + 2 * m + sub));
                    j0 += 64;
                    if (sub) {
                        j0 += (step - 1) * kTok;
                        at += step;
                        s_ph ^= 1;
                    }
                }
                // the next run's queries, once the products of this one have read theirs:
                // its first scores are then on their way while this one's output is written
                t0 += sg.n;
                const Segment *next = run_at(sh, run_idx + 1);
                if (next && m * 128 < next->rows) {
                    // (only a pair that loads may wait here: without its load the barrier
                    // cannot run a phase ahead of the one it waits for)
                    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(bar(kQEmpty), e_ph, abort_flag, a.err));
                    queries(*next);
                }
                e_ph ^= 1;
                // O of the run
                if (mine) {
                    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(bar(kOFull + m), o_ph, abort_flag, a.err));
                    o_ph ^= 1;
                }
                {
                    // the row's sum passes between its two threads
                    float *swap = &sh.top[0][m][0][r];
                    swap[128 * half] = sum;
                    named_bar_sync(pair_bar, 64);
                    sum += swap[128 * (half ^ 1)];
                    named_bar_sync(pair_bar, 64);  // read before the next run writes there
                    // narrow: the second pair hands its maximum, sum and O to the first
                    float mix = 1.0f, mix1 = 0.0f;
                    if (narrow) {
                        if (m == 1 && half == 0) {
                            sh.top[0][1][0][r] = top;
                            sh.top[0][1][1][r] = sum;
                        }
                        tc_fence_before();
                        named_bar_sync(kBarBoth, 512);
                        if (m == 0) {
                            const float top1 = sh.top[0][1][0][r], sum1 = sh.top[0][1][1][r];
                            const float both = fmaxf(top, top1);
                            mix = kv_ex2((top - both) * sl2);
                            mix1 = kv_ex2((top1 - both) * sl2);
                            top = both;
                            sum = sum * mix + sum1 * mix1;
                        }
                    }
                    tc_fence_after();
                    const bool join = narrow && sg.n > 1;
                    const bool writes = live && !(narrow && m == 1);
                    const float inv = sg.whole ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
                    mix *= inv;
                    mix1 *= inv;
                    const size_t o_row = (size_t)(sg.r.q0 + i) * a.q_heads + sg.h * a.group + hh;
                    const int part = sg.i_u0 > c_lo ? 1 : 0;
                    float *slot = a.cta_slots + ((size_t)2 * blockIdx.x + part) * C::kSlot +
                                  ((narrow ? 0 : m * 128) + r) * C::kPitch;
#pragma unroll 1
                    for (int q = 0; q < (narrow && m == 1 ? 0 : D / 64); ++q) {
                        // 32 columns, four V pieces g = 4a..: two groups' 16 dimensions
                        uint32_t o[32];
                        tmem_ld32(o_at + 32 * q, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * mix);
                        if (join) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float o1[16];
                                tmem_ld_32x32b_x16_wait(o_at + 128 + 32 * q + 16 * c, o1);
                                if (mix1 > 0.0f) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        o[16 * c + e] = __float_as_uint(
                                            fmaf(o1[e], mix1, __uint_as_float(o[16 * c + e])));
                                }
                            }
                        }
                        const int at = half * (D / 64) + q, d0 = 64 * (at >> 1) + 16 * (at & 1);
                        if (!writes) continue;
#pragma unroll
                        for (int gr = 0; gr < 2; ++gr) {
                            float x[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                x[e] = __uint_as_float(o[(e >> 2) * 8 + 2 * (e & 3) + gr]);
                            if (sg.whole) {
                                uint32_t y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const __nv_bfloat162 z = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                                    y[e] = *reinterpret_cast<const uint32_t *>(&z);
                                }
                                uint4 *dst = reinterpret_cast<uint4 *>(a.out + o_row * D + d0 + 32 * gr);
                                dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                                dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                            } else {
                                float4 *dst = reinterpret_cast<float4 *>(slot + d0 + 32 * gr);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                            }
                        }
                    }
                    if (writes && half == 0) {
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
                    sh.part_q0[part] = sg.r.q0;
                    sh.part_h[part] = sg.h;
                    sh.part_row0[part] = sg.rt * kRowsItem;
                    sh.part_rows[part] = sg.rows;
                }
                tc_fence_before();  // the reads of O before the next run's first product
                if (narrow) named_bar_sync(kBarBoth, 512);
                run_done(sh, run_idx++);
                run = next;
            }
            fewer_regs<kRegsLaunch>();
            named_bar_sync(kBarRegs, kThreads);
        } else if (w < 24) {
            // ----------------------------------------------- codes to operand tiles --
            fewer_regs<kRegsCodes>();
            if (w < 20)
                unpack_role<D, 0>(a, sh, smem);
            else
                unpack_role<D, 1>(a, sh, smem);
            named_bar_sync(kBarRegs, kThreads);
            more_regs<kRegsLaunch>();
        } else {
            fewer_regs<kRegsMma>();
            // ----------------------------------------------------------------- MMAs --
            // Warp 24 + m issues the products of row tile m.  The tensor pipe holds
            // little more than the instruction it runs, so a warp's waits and commits
            // would leave it idle; two warps fill each other's gaps.
            const int m = w - 24;
            const uint32_t id_s = idesc_f16_m128(kTok / 2);
            const uint32_t id_o = idesc_f16_m128(D) | (1u << 16);  // B N-major
            uint32_t p_ph = 0, q_ph[2] = {0, 0}, t0 = 0;  // t0: tiles of earlier runs
            bool ok = true;
            auto wait = [&](int b, uint32_t ph) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(b), ph, abort_flag, a.err));
                return ok;
            };
            // a tile's slot in the rings of two, and its phase
            auto slot = [&](int k) { return (t0 + k) & 1u; };
            auto phase = [&](int k) { return ((t0 + k) >> 1) & 1u; };
            if (m == 2) {
                Walk walk;
                walk.start(a, sh.prefix, chunks, per_chunk, c_lo, c_hi);
                write_runs(a, sh, walk);
            }
            for (uint32_t run_idx = 0; m < 2 && ok; ++run_idx) {
                const Segment *run = run_at(sh, run_idx);
                if (!run) break;
                const int n = run->n;
                // narrow: warp m takes every other tile, for the same rows, and lets go
                // of a tile for both
                const bool narrow = run->rows <= 128;
                run_done(sh, run_idx);
                const int first = narrow ? m : 0, step = narrow ? 2 : 1;
                const uint32_t q_at = smem + C::kQ + (narrow ? 0u : (uint32_t)m * C::kTileBytes);
                if (!wait(kQFull, q_ph[0])) break;
                q_ph[0] ^= 1;
                if (!narrow) {
                    if (m == 1 && !wait(kQFull + 1, q_ph[1])) break;
                    q_ph[1] ^= 1;
                }
                // the scores of one half of tile k; the tile's second half lets go of it,
                // the run's last one of the queries
                auto scores = [&](int k, uint32_t sub) {
                    mma_qk<D>(s_col(m, sub), q_at, smem + C::kK + slot(k) * C::kTileBytes + sub * (kTok / 2 * 128),
                              id_s);
                    const uint32_t done = sub ? bar(kKEmpty + slot(k)) : 0u;
                    tc_commit2_elect(bar(kSFull + 2 * m + sub), done);
                    if (sub)
                        tc_commit2_elect(narrow ? done : 0u, k + step >= n ? bar(kQEmpty) : 0u);
                };
                if (first < n) {
                    if (!wait(kKFull + slot(first), phase(first))) break;
                    tc_fence_after();
                    scores(first, 0);
                    scores(first, 1);
                    // before the run's first wait for V (the rings' invariant at Bar)
                    if (!wait(kPFull + 2 * m, p_ph)) break;
                } else if (lane == 0) {
                    mbar_arrive(bar(kQEmpty));
                }
                for (int k = first; ok && k < n; k += step) {
                    const bool again = k + step < n;
                    if (!wait(kVFull + slot(k), phase(k))) break;
                    if (again && !wait(kKFull + slot(k + step), phase(k + step))) break;
                    const uint32_t v_at = smem + C::kV + slot(k) * C::kTileBytes, done = bar(kVEmpty + slot(k));
#pragma unroll
                    for (uint32_t sub = 0; sub < 2; ++sub) {
                        if (!wait(kPFull + 2 * m + sub, p_ph)) break;
                        tc_fence_after();
                        mma_pv(o_col(m), s_col(m, sub), v_at + sub * (kTok / 2 * 128), id_o, k > first || sub);
                        tc_commit2_elect(bar(kPv + m), sub ? done : 0u);
                        if (again) scores(k + step, sub);
                    }
                    tc_commit2_elect(narrow ? done : 0u, again ? 0u : bar(kOFull + m));
                    p_ph ^= 1;
                }
                t0 += n;
            }
            named_bar_sync(kBarRegs, kThreads);
            more_regs<kRegsLaunch>();
        }
    }
    if ((w == 24 || w == 25) && __any_sync(0xffffffffu, *(volatile int *)abort_flag)) {
        // products in flight end before the tensor memory is given back
        volatile int none = 0;
        tc_commit_elect(bar(kDrain + w - 24));
        mbar_wait(bar(kDrain + w - 24), 0, &none, a.err);
        __syncwarp();
    }
    tc_fence_before();
    __threadfence();
    __syncthreads();
    tc_fence_after();
    if (w == 27) tmem_dealloc(tmem, kTmemCols);

    // items shared with other CTAs: the last of them adds the parts up
    if (tid < 2) {
        const uint32_t u0 = sh.part_u0[tid], u1 = sh.part_u1[tid];
        bool last = false;
        if (u0 != u1) {
            const uint32_t c0 = u0 / per, c1 = (u1 - 1) / per;
            last = atomicAdd(a.counters + c0, 1) == (int)(c1 - c0);
            if (last) a.counters[c0] = 0;
        }
        sh.last_of[tid] = last;
    }
    __syncthreads();
    for (int part = 0; part < 2; ++part) {
        if (!sh.last_of[part]) continue;
        __threadfence();
        const uint32_t u0 = sh.part_u0[part], c0 = u0 / per, c1 = (sh.part_u1[part] - 1) / per;
        const int q0 = sh.part_q0[part], h = sh.part_h[part], row0 = sh.part_row0[part];
        const int rows = sh.part_rows[part];
        const int odd = u0 > c0 * per ? 1 : 0;  // in its first CTA the item is the last one
        constexpr int kGroup = 2 * (32 / (D / 4));
        for (int row = w * kGroup; row < rows; row += kThreads / 32 * kGroup)
            add_parts<D, 2, 2>(
                (int)(c1 - c0) + 1, row, sl2,
                [&](int i) { return a.cta_slots + ((size_t)2 * (c0 + i) + (i ? 0 : odd)) * C::kSlot; },
                [&](int r, int d4, float mm, float ll, float4 s) {
                    if (r >= rows) return;
                    const int rr = row0 + r, i = div_group(rr, a.gdiv), hh = rr - i * a.group;
                    const size_t o = (size_t)(q0 + i) * a.q_heads + h * a.group + hh;
                    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
                    const __nv_bfloat162 x = __floats2bfloat162_rn(s.x * inv, s.y * inv);
                    const __nv_bfloat162 y = __floats2bfloat162_rn(s.z * inv, s.w * inv);
                    *reinterpret_cast<uint2 *>(a.out + o * D + 4 * d4) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&x),
                                   *reinterpret_cast<const uint32_t *>(&y));
                    if (a.lse && d4 == 0)
                        a.lse[o] = ll > 0.0f ? (mm * sl2 + log2f(ll)) * 0.6931471805599453f : -INFINITY;
                });
    }
}

template <int D>
cudaError_t launch(const KvAttnArgs &a, int grid, cudaStream_t s) {
    static std::atomic<bool> set[64];
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
