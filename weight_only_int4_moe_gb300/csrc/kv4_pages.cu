// Page management of the 4-bit cache (include/moe_kv4.h): taking the lowest free
// pages (reserve, fork), giving them back (free), making the pool dense (compact)
// and copying pages.  A page is free when refs[page] is 0; there is no free list,
// so every call's result follows from refs alone and does not depend on the order
// in which blocks run (the only atomics are adds whose results nobody orders by).
//
// The bookkeeping touches a few bytes per page and is latency: refs are scanned
// from L2.  The bytes are the copies: whole pages (copy, compact) or the live
// tokens of begun ones (fork), streamed as 16-byte loads, eight in flight a lane.
//
// Measured: 200 sequences of up to 4000 tokens in a fragmented pool of 4 layers made
// dense: 210 us for 1.32 GB, 6.3 TB/s (a copy reaches 6.8); 256 branches of 64 sequences
// in 8 layers: 34 us for 144 MB, 4.2 TB/s.  Small pools are
// launches: 10 us for 8 branches (free, take and fork), 6 us for a compaction.  A reserve
// of 256 streams that grow by a token, 16 of them into a new page: 6 us where free pages
// are spread over the pool, of any size; one block scans 4096 pages a turn, so where only
// the last pages are free 27, 101 and 204 us in pools of 100000, 500000 and 2^20 pages.
// Each block of a compaction counts the whole pool: with nothing to move 10, 28 and 93 us.
// Copied pages of 4.6 KB: 6.2 to 6.4 TB/s.
#include "kv4_launch.cuh"

namespace moe {

namespace {

constexpr int kScan = 1024;  // threads of the scanning blocks

// Exclusive prefix sum over the block's kScan threads; total gets the sum.
MOE_DEV int block_scan(int v, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    if (w == 0) {
        int y = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        warp_sums[lane] = y;
    }
    __syncthreads();
    total = warp_sums[kScan / 32 - 1];
    const int before = w ? warp_sums[w - 1] : 0;
    __syncthreads();
    return before + x - v;
}

MOE_DEV int block_sum(int v, int *warp_sums) {
    int total;
    block_scan(v, warp_sums, total);
    return total;
}

// ------------------------------------------------------------ reserve, fork --
// Scratch: [0] pages found, [16 + i] first rank of request i's pages (-1:
// skipped), [16 + n + i] how many it needs, then the page of each rank.
struct TakeArgs {
    KvPages p;
    moe_kv4_seqs q;
    const int32_t *a, *b;  // fork: parents, children; reserve: ids, new lengths
    int fork, n;
    int32_t *scratch;
    uint32_t *err;
};

// Pages of len tokens (any len up to the largest int).
MOE_DEV int pages_for(int len, int ps) { return len / ps + (len % ps > 0); }

// Requests may ask for more pages than an int counts.  What the pool cannot hold fails
// whatever its exact size, so a request's need and the running total are cut off at one
// page more than there are, and the sum of a turn's kScan needs stays below 2^31.
__global__ void __launch_bounds__(kScan) kv4_take_kernel(const TakeArgs t) {
    __shared__ int warp_sums[32];
    pdl_wait();
    const int ps = t.p.ps, n = t.n;
    int32_t *first = t.scratch + 16, *need_of = first + n, *page_of = need_of + n;
    int total = 0;
    for (int i0 = 0; i0 < n; i0 += kScan) {
        const int i = i0 + threadIdx.x;
        int need = 0;
        bool ok = false;
        if (i < n) {
            const int x = t.a[i];
            ok = (unsigned)x < (unsigned)t.q.seqs;
            const int len = ok ? t.q.lens[x] : 0;
            if (t.fork) {
                const int c = t.b[i];
                ok = ok && (unsigned)c < (unsigned)t.q.seqs && c != x && t.q.lens[c] == 0 &&
                     len >= 0 && len <= t.q.table_stride * (long long)ps;
                need = ok && len % ps != 0;
            } else {
                const int to = t.b[i];
                ok = ok && len >= 0 && to >= len && to <= t.q.table_stride * (long long)ps;
                need = ok ? min(pages_for(to, ps) - pages_for(len, ps), t.p.n_pages + 1) : 0;
            }
            if (!ok) kv_report(t.err, MOE_KV4_DEVERR_SEQ);
        }
        int sum;
        const int at = total + block_scan(need, warp_sums, sum);
        if (i < n) {
            first[i] = ok ? at : -1;
            need_of[i] = need;
        }
        total = min(total + sum, t.p.n_pages + 1);
    }
    // the lowest free pages
    int found = 0;
    for (int p0 = 0; p0 < t.p.n_pages && found < total; p0 += 4 * kScan) {
        const int p = p0 + 4 * threadIdx.x;
        bool f[4];
        int c = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            f[u] = p + u < t.p.n_pages && t.q.refs[p + u] == 0;
            c += f[u];
        }
        int sum;
        int r = found + block_scan(c, warp_sums, sum);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (f[u]) {
                if (r < total) page_of[r] = p + u;
                ++r;
            }
        found += sum;
    }
    if (threadIdx.x == 0) t.scratch[0] = found;
    if (t.fork) return;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < n; i += kScan / 32) {
        const int r = first[i], need = need_of[i];
        if (r < 0) continue;
        if (r + need > found) {
            if (lane == 0) kv_report(t.err, MOE_KV4_DEVERR_NO_PAGES);
            continue;
        }
        const int x = t.a[i], to = t.b[i];
        int32_t *row = t.q.tables + (size_t)x * t.q.table_stride + pages_for(to, ps) - need;
        for (int j = lane; j < need; j += 32) {
            const int page = page_of[r + j];
            row[j] = page;
            t.q.refs[page] = 1;
        }
        if (lane == 0) t.q.lens[x] = to;
    }
}

// A fork's second half: blocks 0..n-1 copy a table row each and count the shared
// pages; each warp of the others copies the begun page's live tokens of one
// (request, layer, head).
__global__ void __launch_bounds__(256) kv4_fork_kernel(const TakeArgs t) {
    pdl_wait();
    const int ps = t.p.ps, n = t.n;
    const int found = t.scratch[0];
    const int32_t *first = t.scratch + 16, *need_of = first + n, *page_of = need_of + n;
    if (blockIdx.x < n) {
        const int i = blockIdx.x, r = first[i], need = need_of[i];
        if (r < 0) return;
        if (r + need > found) {
            if (threadIdx.x == 0) kv_report(t.err, MOE_KV4_DEVERR_NO_PAGES);
            return;
        }
        const int x = t.a[i], c = t.b[i], len = t.q.lens[x], full = len / ps;
        const int32_t *src = t.q.tables + (size_t)x * t.q.table_stride;
        int32_t *dst = t.q.tables + (size_t)c * t.q.table_stride;
        for (int j = threadIdx.x; j < full; j += blockDim.x) {
            const int page = src[j];
            dst[j] = page;
            if ((unsigned)page < (unsigned)t.p.n_pages)
                atomicAdd(t.q.refs + page, 1);
            else
                kv_report(t.err, MOE_KV4_DEVERR_PAGE);
        }
        if (threadIdx.x == 0) {
            if (need) {
                dst[full] = page_of[r];
                t.q.refs[page_of[r]] = 1;
            }
            t.q.lens[c] = len;
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const long long task = (long long)(blockIdx.x - n) * 8 + (threadIdx.x >> 5);
    const int per = t.p.layers * t.p.hkv;
    const int i = (int)(task / per), rest = (int)(task % per);
    if (i >= n) return;
    const int r = first[i];
    if (r < 0 || !need_of[i] || r + 1 > found) return;
    const int x = t.a[i], len = t.q.lens[x], live = len % ps, D = t.p.D;
    const int old = t.q.tables[(size_t)x * t.q.table_stride + len / ps];
    if ((unsigned)old >= (unsigned)t.p.n_pages) {
        if (lane == 0) kv_report(t.err, MOE_KV4_DEVERR_PAGE);
        return;
    }
    const size_t layer = (size_t)(rest / t.p.hkv) * t.p.n_pages;
    const int head = rest % t.p.hkv;
    const uint8_t *s = t.p.pages + ((layer + old) * t.p.hkv + head) * t.p.block;
    uint8_t *d = t.p.pages + ((layer + page_of[r]) * t.p.hkv + head) * t.p.block;
    // codes: two runs of live rows of D / 2 bytes; scales: two of live * D / 16 bytes
    const int c16 = live * (D / 32), vofs = ps * (D / 2);
    uint4 v[8];
    for (int u0 = lane; u0 < 2 * c16; u0 += 256) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int e = u0 + 32 * u;
            if (e < 2 * c16)
                v[u] = *reinterpret_cast<const uint4 *>(s + (e < c16 ? 16 * e : vofs + 16 * (e - c16)));
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int e = u0 + 32 * u;
            if (e < 2 * c16)
                *reinterpret_cast<uint4 *>(d + (e < c16 ? 16 * e : vofs + 16 * (e - c16))) = v[u];
        }
    }
    const int s4 = live * (D / 64), sofs = ps * D, sv = ps * (D / 16);
    for (int e = lane; e < 2 * s4; e += 32) {
        const int o = sofs + (e < s4 ? 4 * e : sv + 4 * (e - s4));
        *reinterpret_cast<uint32_t *>(d + o) = *reinterpret_cast<const uint32_t *>(s + o);
    }
}

// --------------------------------------------------------------------- free --
__global__ void __launch_bounds__(128) kv4_free_kernel(const KvPages p, const moe_kv4_seqs q,
                                                       const int32_t *ids, uint32_t *err) {
    pdl_wait();
    const int x = ids[blockIdx.x];
    if ((unsigned)x >= (unsigned)q.seqs) {
        if (threadIdx.x == 0) kv_report(err, MOE_KV4_DEVERR_SEQ);
        return;
    }
    const int n = min(pages_for(q.lens[x], p.ps), q.table_stride);
    int32_t *row = q.tables + (size_t)x * q.table_stride;
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
        const int page = row[j];
        row[j] = -1;
        if ((unsigned)page >= (unsigned)p.n_pages) {
            kv_report(err, MOE_KV4_DEVERR_PAGE);
        } else if (atomicSub(q.refs + page, 1) <= 0) {
            atomicAdd(q.refs + page, 1);
            kv_report(err, MOE_KV4_DEVERR_SEQ);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) q.lens[x] = 0;
}

// ----------------------------------------------------------- copy, compact --
// One warp copies up to 256 16-byte units, eight loads in flight a lane.
MOE_DEV void copy_run(const uint4 *s, uint4 *d, int n) {
    const int lane = threadIdx.x & 31;
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
        if (lane + 32 * u < n) v[u] = s[lane + 32 * u];
#pragma unroll
    for (int u = 0; u < 8; ++u)
        if (lane + 32 * u < n) d[lane + 32 * u] = v[u];
}

// Copies page src[i] to dst[i] in every layer for i < n, the grid's warps taking
// runs in turn.
MOE_DEV void copy_pages(const KvPages &p, const int32_t *src, const int32_t *dst, int n,
                        uint32_t *err) {
    const int units = (int)((size_t)p.hkv * p.block / 16), runs = (units + 255) / 256;
    const long long tasks = (long long)n * p.layers * runs;
    const int warps = gridDim.x * (blockDim.x >> 5);
    for (long long k = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); k < tasks; k += warps) {
        const int run = (int)(k % runs);
        const long long m = k / runs;
        const int layer = (int)(m % p.layers), i = (int)(m / p.layers);
        const int a = src[i], b = dst[i];
        if (a < 0 || b < 0) continue;
        if (a >= p.n_pages || b >= p.n_pages) {
            if (layer == 0 && run == 0 && (threadIdx.x & 31) == 0)
                kv_report(err, MOE_KV4_DEVERR_PAGE);
            continue;
        }
        const size_t base = (size_t)layer * p.n_pages;
        const uint4 *s = reinterpret_cast<const uint4 *>(p.pages) + (base + a) * units + run * 256;
        uint4 *d = reinterpret_cast<uint4 *>(p.pages) + (base + b) * units + run * 256;
        copy_run(s, d, min(256, units - run * 256));
    }
}

__global__ void __launch_bounds__(256) kv4_copy_kernel(const KvPages p, const int32_t *src,
                                                       const int32_t *dst, int n, uint32_t *err) {
    pdl_wait();
    copy_pages(p, src, dst, n, err);
}

// Scratch of compact: [0] moves, [1] pages in use; from 16: the moves' sources,
// their targets, and each source page's move.
struct CompactArgs {
    KvPages p;
    moe_kv4_seqs q;
    int32_t *tables_out, *refs_out, *n_used, *scratch;
    uint32_t *err;
};

// Each block lists the moves of 4096 pages; every block counts the whole of refs
// for itself (a few loads a thread from L2, and no second launch).
__global__ void __launch_bounds__(kScan) kv4_moves_kernel(const CompactArgs c) {
    __shared__ int warp_sums[32];
    pdl_wait();
    const int n = c.p.n_pages, lo = blockIdx.x * 4 * kScan;
    int32_t *src = c.scratch + 16, *dst = src + n, *move_of = dst + n;
    int all = 0, before = 0;
    for (int p = threadIdx.x; p < n; p += kScan) {
        const int u = c.q.refs[p] > 0;
        all += u;
        before += p < lo ? u : 0;
    }
    const int used = block_sum(all, warp_sums);
    before = block_sum(before, warp_sums);
    int low = 0;  // pages in use that stay
    for (int p = threadIdx.x; p < used; p += kScan) low += c.q.refs[p] > 0;
    low = block_sum(low, warp_sums);
    const int p = lo + 4 * threadIdx.x;
    bool f[4];
    int k = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        f[u] = p + u < n && c.q.refs[p + u] > 0;
        k += f[u];
    }
    int sum;
    int r = before + block_scan(k, warp_sums, sum);  // pages in use below p
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int e = p + u;
        if (e < n) {
            if (f[u] && e >= used) {
                src[r - low] = e;
                move_of[e] = r - low;
            }
            if (!f[u] && e < used) dst[e - r] = e;
            r += f[u];
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        c.scratch[0] = used - low;
        c.scratch[1] = used;
        *c.n_used = used;
    }
}

__global__ void __launch_bounds__(256) kv4_compact_kernel(const CompactArgs c) {
    pdl_wait();
    const int n = c.p.n_pages, moves = c.scratch[0], used = c.scratch[1];
    const int32_t *src = c.scratch + 16, *dst = src + n, *move_of = dst + n;
    const int threads = gridDim.x * blockDim.x, id = blockIdx.x * blockDim.x + threadIdx.x;
    // refs: a target takes its source's count and clears it, whoever else stays
    // keeps its own (the two never touch the same entry, so refs_out may be refs)
    for (int i = id; i < moves; i += threads) {
        const int count = c.q.refs[src[i]];
        c.refs_out[dst[i]] = count;
        c.refs_out[src[i]] = 0;
    }
    if (c.refs_out != c.q.refs)
        for (int p = id; p < n; p += threads) {
            const int r = c.q.refs[p];
            if (p < used ? r > 0 : r <= 0) c.refs_out[p] = max(r, 0);
        }
    const long long entries = (long long)c.q.seqs * c.q.table_stride;
    for (long long e = id; e < entries; e += threads) {
        const int page = c.q.tables[e];
        int to = page;
        if (page >= used && page < n) {
            const int m = move_of[page];
            // an entry whose page nobody counts (refs 0) has no move
            to = (unsigned)m < (unsigned)moves && src[m] == page ? dst[m] : page;
        }
        c.tables_out[e] = to;
    }
    copy_pages(c.p, src, dst, moves, c.err);
}

cudaLaunchConfig_t config(long long grid, unsigned block, cudaStream_t s, cudaLaunchAttribute &at) {
    auto c = pdl_config((unsigned)(grid < 1 ? 1 : grid), block, 0, s);
    c.numAttrs = pdl_attr(at);
    c.attrs = &at;
    return c;
}

}  // namespace

cudaError_t launch_kv4_take(const KvPages &p, const moe_kv4_seqs &q, const int32_t *a,
                            const int32_t *b, bool fork, int n, void *scratch, uint32_t *err,
                            cudaStream_t s) {
    TakeArgs t{p, q, a, b, fork, n, reinterpret_cast<int32_t *>(scratch), err};
    cudaLaunchAttribute at{};
    auto c = config(1, kScan, s, at);
    cudaError_t e = cudaLaunchKernelEx(&c, kv4_take_kernel, t);
    if (e != cudaSuccess || !fork) return e;
    c = config(n + ((long long)n * p.layers * p.hkv + 7) / 8, 256, s, at);
    return cudaLaunchKernelEx(&c, kv4_fork_kernel, t);
}

cudaError_t launch_kv4_free(const KvPages &p, const moe_kv4_seqs &q, const int32_t *ids, int n,
                            uint32_t *err, cudaStream_t s) {
    cudaLaunchAttribute at{};
    auto c = config(n, 128, s, at);
    return cudaLaunchKernelEx(&c, kv4_free_kernel, p, q, ids, err);
}

cudaError_t launch_kv4_compact(const KvPages &p, const moe_kv4_seqs &q, int32_t *tables_out,
                               int32_t *refs_out, int32_t *n_used, void *scratch, uint32_t *err,
                               int sms, cudaStream_t s) {
    CompactArgs a{p, q, tables_out, refs_out, n_used, reinterpret_cast<int32_t *>(scratch), err};
    cudaLaunchAttribute at{};
    auto c = config((p.n_pages + 4 * kScan - 1) / (4 * kScan), kScan, s, at);
    cudaError_t e = cudaLaunchKernelEx(&c, kv4_moves_kernel, a);
    if (e != cudaSuccess) return e;
    c = config(8ll * sms, 256, s, at);
    return cudaLaunchKernelEx(&c, kv4_compact_kernel, a);
}

cudaError_t launch_kv4_copy(const KvPages &p, const int32_t *src, const int32_t *dst, int n,
                            uint32_t *err, int sms, cudaStream_t s) {
    const long long runs = ((long long)p.hkv * p.block / 16 + 255) / 256 * p.layers * n;
    cudaLaunchAttribute at{};
    auto c = config(runs < 64ll * sms ? (runs + 7) / 8 : 8ll * sms, 256, s, at);
    return cudaLaunchKernelEx(&c, kv4_copy_kernel, p, src, dst, n, err);
}

}  // namespace moe
