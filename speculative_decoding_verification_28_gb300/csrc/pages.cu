// pages.cu -- the book of a page pool: which pages a sequence has (table,
// held), how often each is named (refs), and copies of whole pages.
//
// fork, reserve and compact are a few kB of integers, so a latency: one CTA
// walks the pool's refs in order (4 bytes a page, 16384 pages a step), which
// makes "the lowest free page first" a prefix sum and every result independent
// of the order in which threads run.  Only sums into refs are atomic, and
// those commute.  A barrier orders what a CTA does to global memory for its own
// threads, atomics (read past L1) among it; fences for the device beside them
// cost reserve 2 of 10.5 us.  The copies are bound by HBM.
#include <limits.h>

#include "paged.h"
#include "spec_common.cuh"

namespace spec {

constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kPerThread = 16;  // pages of a thread in a step
constexpr int kForkThreads = 256;
// Table entries of a call that one CTA goes through in one launch, which is 1.8 us less for
// the caller: forks of 16 rows of 64 pages 8.4 us a call (3.8 on the device), in two launches
// 10.1 (3.9), but of 64 rows 7.8 on the device against 4.4; tables of 64 rows of 64 compacted
// 8.0 a call (6.7), 9.9 (6.9), of 256 rows 14.5 (13.6), 14.4 (10.4).
constexpr int kForkOne = 1024, kCompactOne = 4096;

__host__ __device__ __forceinline__ long long pages_for(long long tokens, int page_log2)
{
    return (tokens + (1ll << page_log2) - 1) >> page_log2;
}
__device__ __forceinline__ bool in_pool(const PagesArgs &p, int page) { return page >= 0 && page < p.P; }

size_t page_workspace(int B, int MP, int P)
{
    const size_t fork = (size_t)B * ((size_t)MP + 1), reserve = 6 * (size_t)B + 3 * (size_t)P, compact = 3 * (size_t)P + 1;
    const size_t most = fork > reserve ? fork : reserve;
    return align256((most > compact ? most : compact) * 4);
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// Every sequence reads its source's row as it was before the call, so the new
// rows wait in the workspace ([B, MP], then [B] pages or -1: refused) until all
// have been read.  THREADS of sequence b, a warp or a CTA; t: which of them.
template <int THREADS>
__device__ __forceinline__ void fork_read(const ForkArgs &a, int b, int t)
{
    const PagesArgs &p = a.p;
    const int dst = a.dst ? a.dst[b] : b, src = a.src[b];
    bool ok = dst >= 0 && dst < p.N && src >= -1 && src < p.N;
    int n = 0, had = 0;
    if (ok) {
        had = p.held[dst];
        ok = had >= 0 && had <= p.MP;
        if (src >= 0) {
            const int has = p.held[src];
            const long long want = a.length ? pages_for(a.length[b], p.page_log2) : has;
            ok = ok && has >= 0 && has <= p.MP && (!a.length || a.length[b] >= 0) && want <= has;
            n = ok ? (int)want : 0;
        }
    }
    const bool twice = repeated_row(a.dst, p.B, dst);
    ok = ok && !twice;
    if (ok) {
        for (int i = t; i < n; i += THREADS)
            ok &= in_pool(p, p.table[(size_t)src * p.MP + i]);
        for (int i = t; i < had; i += THREADS)
            ok &= in_pool(p, p.table[(size_t)dst * p.MP + i]);
    }
    ok = THREADS == 32 ? __all_sync(0xFFFFFFFFu, ok) : __syncthreads_and(ok);
    if (t == 0) {
        p.ws[(size_t)p.B * p.MP + b] = ok ? n : -1;
        if (p.flags)
            p.flags[b] = ok ? 0u : SPEC_FLAG_BAD_STATE;
    }
    if (!ok)
        return;
    for (int i = t; i < p.MP; i += THREADS) {
        const int page = i < n ? p.table[(size_t)src * p.MP + i] : -1;
        p.ws[(size_t)b * p.MP + i] = page;
        if (i < n)
            atomicAdd(p.refs + page, 1);
        if (i < had)
            atomicSub(p.refs + p.table[(size_t)dst * p.MP + i], 1);
    }
}
template <int THREADS>
__device__ __forceinline__ void fork_write(const ForkArgs &a, int b, int t)
{
    const PagesArgs &p = a.p;
    const int n = p.ws[(size_t)p.B * p.MP + b];
    if (n < 0)
        return;
    const int dst = a.dst ? a.dst[b] : b;
    for (int i = t; i < p.MP; i += THREADS)
        p.table[(size_t)dst * p.MP + i] = p.ws[(size_t)b * p.MP + i];
    if (t == 0)
        p.held[dst] = n;
}

__global__ void __launch_bounds__(kForkThreads) fork_read_kernel(const ForkArgs a)
{
    fork_read<kForkThreads>(a, blockIdx.x, threadIdx.x);
}
__global__ void __launch_bounds__(kForkThreads) fork_write_kernel(const ForkArgs a)
{
    fork_write<kForkThreads>(a, blockIdx.x, threadIdx.x);
}
// Both in one launch, a warp a sequence.
__global__ void __launch_bounds__(kBookThreads) fork_small_kernel(const ForkArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int b = warp; b < a.p.B; b += kBookWarps)
        fork_read<32>(a, b, lane);
    __syncthreads();
    for (int b = warp; b < a.p.B; b += kBookWarps)
        fork_write<32>(a, b, lane);
}

cudaError_t launch_page_fork(const ForkArgs &a, cudaStream_t st)
{
    if ((long long)a.p.B * a.p.MP <= kForkOne) {
        fork_small_kernel<<<1, kBookThreads, 0, st>>>(a);
    } else {
        fork_read_kernel<<<a.p.B, kForkThreads, 0, st>>>(a);
        fork_write_kernel<<<a.p.B, kForkThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// walking the pool in order
// ---------------------------------------------------------------------------
// exclusive prefix of v over the block and its total; `s`: a word per warp.
// Every thread calls; barriers on both sides.  MOST: where sums stop, for values
// up to it (what lies behind one that stopped is then no prefix any more).
template <int MOST = INT_MAX>
__device__ __forceinline__ int block_before(int v, int *s, int *total)
{
    static_assert(MOST == INT_MAX || MOST <= INT_MAX / 2, "two sums in 31 bits");
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, x, m);
        if (lane >= m)
            x = min(x + o, MOST);
    }
    __syncthreads();
    if (lane == 31)
        s[w] = x;
    __syncthreads();
    int y = s[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, y, m);
        if (lane >= m)
            y = min(y + o, MOST);
    }
    *total = __shfl_sync(0xFFFFFFFFu, y, 31);
    const int warps = __shfl_sync(0xFFFFFFFFu, y, w) - s[w];
    return warps + x - v;
}
static_assert(kBookWarps == 32, "a lane per warp's word");

// Bits of this thread's pages p0 .. p0 + 15 that are live; beyond the pool: none.
__device__ __forceinline__ uint32_t live_bits(const PagesArgs &p, int p0)
{
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
        if (p0 + i < p.P && __ldcg(p.refs + p0 + i) > 0)
            bits |= 1u << i;
    return bits;
}
__device__ __forceinline__ uint32_t page_bits(const PagesArgs &p, int p0)
{
    const int n = min(kPerThread, max(0, p.P - p0));
    return (1u << n) - 1;
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
constexpr int kMostWishes = 1 << 29;  // that are counted
constexpr int kWishes = 1024;     // sequences whose wishes fit in shared memory
constexpr int kWishLanes = 8;     // threads of a sequence

// What the sequences want, by sequence: of row's h pages those at places lo .. hi - 1 are
// written, and it ends with n; h < 0: refused.  at: first the pages it needs, then the place
// of the first of them among all.
struct Wishes {
    int *row, *lo, *hi, *n, *h, *at;
    __device__ Wishes(int *p, int B) : row(p), lo(p + B), hi(lo + B), n(hi + B), h(n + B), at(h + B) {}
};

// An entry that will be replaced holds ~page until it is.
__global__ void __launch_bounds__(kBookThreads) reserve_kernel(const ReserveArgs a)
{
    __shared__ int s_words[32];
    __shared__ int s_wishes[6 * kWishes];
    const PagesArgs &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // eight threads a sequence: their lane among them, their bits in the warp
    const int k = lane & (kWishLanes - 1), shift = lane & ~(kWishLanes - 1);
    const unsigned us = ((1u << kWishLanes) - 1) << shift;
    constexpr int kGroups = kBookThreads / kWishLanes;
    const int first_b = tid / kWishLanes;
    int *grant = p.ws, *writers = grant + p.P, *last = writers + p.P;
    const Wishes w(p.B <= kWishes ? s_wishes : last + p.P, p.B);

    // rows named twice
    for (int b = warp; b < p.B; b += kBookWarps) {
        const int row = a.idx ? a.idx[b] : b;
        const bool twice = repeated_row(a.idx, p.B, row);
        if (lane == 0) {
            w.row[b] = row;
            w.h[b] = twice ? -1 : 0;
        }
    }
    __syncthreads();
    // check, and let go of pages behind the new end
    for (int b = first_b; b < p.B; b += kGroups) {
        const int row = w.row[b];
        const long long first = a.first[b], total = a.total[b], n = pages_for(total, p.page_log2);
        bool ok = w.h[b] == 0 && row >= 0 && row < p.N && first >= 0 && total >= 0 && n <= p.MP;
        const int h = ok ? p.held[row] : 0;
        ok = ok && h >= 0 && h <= p.MP;
        const int keep = (int)(h < n ? h : n);
        const long long from = first < total ? first >> p.page_log2 : keep;
        const int lo = from < keep ? (int)from : keep;
        int32_t *entries = p.table + (size_t)(ok ? row : 0) * p.MP;
        if (ok)
#pragma unroll 4
            for (int i = lo + k; i < h; i += kWishLanes)
                ok &= in_pool(p, entries[i]);
        ok = __all_sync(us, ok);
        if (ok) {
            for (int i = lo + k; i < keep; i += kWishLanes) {
                writers[entries[i]] = 0;
                last[entries[i]] = -1;
            }
#pragma unroll 4
            for (int i = (int)n + k; i < h; i += kWishLanes) {
                atomicSub(p.refs + entries[i], 1);
                entries[i] = -1;
            }
        }
        __syncwarp(us);
        if (k == 0) {
            w.lo[b] = lo;
            w.hi[b] = ok ? keep : lo;
            w.n[b] = ok ? (int)n : 0;
            w.h[b] = ok ? h : -1;
            if (p.flags)
                p.flags[b] = ok ? 0u : SPEC_FLAG_BAD_STATE;
            a.copies[2 * b] = -1;
            a.copies[2 * b + 1] = -1;
        }
    }
    __syncthreads();
    // how many will write a page that several name, and which is the last of them
    for (int b = first_b; b < p.B; b += kGroups)
        for (int i = w.lo[b] + k; i < w.hi[b]; i += kWishLanes) {
            const int page = p.table[(size_t)w.row[b] * p.MP + i];
            if (__ldcg(p.refs + page) > 1) {
                atomicAdd(writers + page, 1);
                atomicMax(last + page, b);
            }
        }
    __syncthreads();
    // Each of them takes another page, but the last where nobody else names it.
    for (int b = first_b; b < p.B; b += kGroups) {
        int need = 0;
        for (int i = w.lo[b] + k; i < w.hi[b]; i += kWishLanes) {
            int32_t *e = p.table + (size_t)w.row[b] * p.MP + i;
            const int page = *e, refs = __ldcg(p.refs + page);
            if (refs > 1 && !(__ldcg(writers + page) == refs && __ldcg(last + page) == b)) {
                *e = ~page;
                ++need;
            }
        }
        need = __reduce_add_sync(us, need);
        if (k == 0)
            w.at[b] = w.h[b] < 0 ? 0 : need + max(0, w.n[b] - w.h[b]);
        __syncwarp(us);
    }
    __syncthreads();

    // places of the sequences' wishes, in order
    int total = 0;
    for (int c = 0; c < p.B; c += kBookThreads) {
        const int b = c + tid, v = b < p.B ? w.at[b] : 0;
        int sum;
        const int before = block_before<kMostWishes>(v, s_words, &sum);
        if (b < p.B)
            w.at[b] = total + before;
        total = min(total + sum, kMostWishes);  // far more than there can be
    }
    // the lowest free pages
    int found = 0;
    for (int c = 0; c < p.P && found < total; c += kBookThreads * kPerThread) {
        const int p0 = c + tid * kPerThread;
        uint32_t free = page_bits(p, p0) & ~live_bits(p, p0);
        int sum;
        int at = found + block_before(__popc(free), s_words, &sum);
        for (; free && at < total; free &= free - 1, ++at)
            grant[at] = p0 + __ffs(free) - 1;
        found += sum;
    }
    const bool enough = found >= total;
    if (tid == 0)
        *a.missing = enough ? 0 : total - found;
    __syncthreads();

    for (int b = first_b; b < p.B; b += kGroups) {
        if (w.h[b] < 0)
            continue;
        const int row = w.row[b], hi = w.hi[b], n = w.n[b], first = a.first[b];
        int at = w.at[b];
        for (int c = w.lo[b]; c < (enough ? n : hi); c += kWishLanes) {
            const int i = c + k;
            int32_t *e = p.table + (size_t)row * p.MP + (i < n ? i : 0);
            const int old = i < hi ? *e : 0;
            const bool fresh = i < n && (i < hi ? old < 0 : enough);
            const unsigned all = __ballot_sync(us, fresh && enough) >> shift;
            if (fresh && !enough)
                *e = ~old;  // as it was
            if (fresh && enough) {
                const int page = grant[at + __popc(all & ((1u << k) - 1))];
                *e = page;
                p.refs[page] = 1;
                if (i < hi) {
                    atomicSub(p.refs + ~old, 1);
                    if (i == first >> p.page_log2 && (first & ((1 << p.page_log2) - 1))) {
                        a.copies[2 * b] = ~old;
                        a.copies[2 * b + 1] = page;
                    }
                }
            }
            at += __popc(all);
        }
        if (k == 0)
            p.held[row] = enough ? n : hi;
    }
}

cudaError_t launch_page_reserve(const ReserveArgs &a, cudaStream_t st)
{
    reserve_kernel<<<1, kBookThreads, 0, st>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// With n live pages, the r-th live page from n on goes to the r-th free one
// below n.  Workspace: [P] free ones, [P] live ones, [P] new places (from n on), n.
template <int THREADS>
__device__ __forceinline__ void rename_row(const PagesArgs &p, const int *place, int row, int t)
{
    const int live = place[p.P], n = min(p.held[row], p.MP);
    for (int i = t; i < n; i += THREADS) {
        int32_t *e = p.table + (size_t)row * p.MP + i;
        if (*e >= live && *e < p.P)
            *e = place[*e];
    }
}
// RENAME: the tables too
template <bool RENAME>
__global__ void __launch_bounds__(kBookThreads) compact_kernel(const CompactArgs a)
{
    __shared__ int s_words[32];
    const PagesArgs &p = a.p;
    const int tid = threadIdx.x;
    int *hole = p.ws, *mover = hole + p.P, *place = mover + p.P;
    int live = 0;
    for (int c = 0; c < p.P; c += kBookThreads * kPerThread) {
        int sum;
        block_before(__popc(live_bits(p, c + tid * kPerThread)), s_words, &sum);
        live += sum;
    }
    int holes = 0, movers = 0;
    for (int c = 0; c < p.P; c += kBookThreads * kPerThread) {
        const int p0 = c + tid * kPerThread;
        const uint32_t bits = live_bits(p, p0), all = page_bits(p, p0);
        const uint32_t low = p0 >= live ? 0u : live - p0 >= kPerThread ? ~0u : (1u << (live - p0)) - 1;
        uint32_t up = bits & ~low, empty = all & ~bits & low;
        int sum;
        int at = block_before(__popc(up) << 16 | __popc(empty), s_words, &sum);
        int h = holes + (at & 0xFFFF), m = movers + (at >> 16);
        for (; empty; empty &= empty - 1)
            hole[h++] = p0 + __ffs(empty) - 1;
        for (uint32_t rest = all & ~low; rest; rest &= rest - 1) {
            const int page = p0 + __ffs(rest) - 1;
            if (bits >> (page - p0) & 1)
                mover[m++] = page;
            else
                place[page] = page;
        }
        holes += sum & 0xFFFF;
        movers += sum >> 16;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kBookThreads) {
        const int from = mover[i], to = hole[i];
        a.moves[2 * i] = from;
        a.moves[2 * i + 1] = to;
        place[from] = to;
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
    }
    if (tid == 0) {
        *a.n_moves = movers;
        place[p.P] = live;
    }
    if (!RENAME)
        return;
    __syncthreads();
    for (int row = tid >> 5; row < p.N; row += kBookWarps)
        rename_row<32>(p, place, row, tid & 31);
}

__global__ void __launch_bounds__(kForkThreads) rename_kernel(const CompactArgs a)
{
    rename_row<kForkThreads>(a.p, a.p.ws + 2 * (size_t)a.p.P, blockIdx.x, threadIdx.x);
}

cudaError_t launch_page_compact(const CompactArgs &a, cudaStream_t st)
{
    if ((long long)a.p.N * a.p.MP <= kCompactOne) {
        compact_kernel<true><<<1, kBookThreads, 0, st>>>(a);
    } else {
        compact_kernel<false><<<1, kBookThreads, 0, st>>>(a);
        rename_kernel<<<a.p.N, kForkThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 8;  // 16-byte words of a thread in flight
static_assert(kCopyChunk == kCopyThreads * kCopyEach * 16, "what the host counts a page's chunks by");

// CTA (x, y): chunk x of a page, the chunks of all slabs numbered through, of every
// gridDim.y-th pair.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PageCopyArgs a, int chunks, int chunk_bytes)
{
    const int n = a.n_pairs ? max(0, min(*a.n_pairs, a.M)) : a.M;
    if (blockIdx.x == 0 && blockIdx.y == 0 && a.err) {
        int bad = 0;
        for (int c = 0; c < n; c += kCopyThreads) {
            const int i = c + threadIdx.x;
            const int from = i < n ? a.pairs[2 * i] : -1, to = i < n ? a.pairs[2 * i + 1] : -1;
            bad += __syncthreads_count(from != -1 && (from < 0 || from >= a.P || to < 0 || to >= a.P));
        }
        if (threadIdx.x == 0)
            *a.err = bad;
    }
    if (chunks == 0)
        return;
    const int slab = blockIdx.x / chunks, chunk = blockIdx.x - slab * chunks;
    const long long off = (long long)chunk * chunk_bytes;
    unsigned char *base = a.pool + (long long)slab * a.P * a.bytes + off;
    const int words = (int)(min((long long)chunk_bytes, a.bytes - off) / 16);
    const int2 *pairs = reinterpret_cast<const int2 *>(a.pairs);
    int i = blockIdx.y;
    const bool wide = reinterpret_cast<uintptr_t>(a.pairs) % 8 == 0;
    auto pair_at = [&](int j) {
        return j >= n ? make_int2(-1, -1) : wide ? __ldg(pairs + j) : make_int2(a.pairs[2 * j], a.pairs[2 * j + 1]);
    };
    int2 next = pair_at(i);
    for (; i < n; i += gridDim.y) {
        const int from = next.x, to = next.y;
        next = pair_at(i + gridDim.y);
        if (from < 0 || from >= a.P || to < 0 || to >= a.P)
            continue;
        const uint4 *src = reinterpret_cast<const uint4 *>(base + from * a.bytes);
        uint4 *dst = reinterpret_cast<uint4 *>(base + to * a.bytes);
        uint4 x[kCopyEach];
#pragma unroll
        for (int k = 0; k < kCopyEach; ++k)
            if (k * kCopyThreads + threadIdx.x < words)
                x[k] = src[k * kCopyThreads + threadIdx.x];
#pragma unroll
        for (int k = 0; k < kCopyEach; ++k)
            if (k * kCopyThreads + threadIdx.x < words)
                dst[k * kCopyThreads + threadIdx.x] = x[k];
    }
}

cudaError_t launch_page_copy(const PageCopyArgs &a, cudaStream_t st)
{
    // chunks of a page, as even as 16-byte words allow
    const int chunks = (int)copy_chunks(a.bytes);
    const long long words = a.bytes / 16, each = (words + chunks - 1) / chunks;
    const long long x = (long long)a.slabs * chunks, most = 8 * kSms;  // eight CTAs an SM
    const long long y = x < 1 ? 1 : most / x < 1 ? 1 : most / x < a.M ? most / x : a.M > 0 ? a.M : 1;
    page_copy_kernel<<<dim3((unsigned)(x < 1 ? 1 : x), (unsigned)y), kCopyThreads, 0, st>>>(a, x < 1 ? 0 : chunks,
                                                                                           (int)(each * 16));
    return cudaGetLastError();
}

}  // namespace spec
