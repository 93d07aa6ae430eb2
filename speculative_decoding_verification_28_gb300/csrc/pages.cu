// pages.cu -- the book of a page pool: which pages a sequence has (table,
// held), how often each is named (refs), and copies of whole pages.
//
// fork, reserve and compact are a few kB of integers, so a latency: one CTA
// walks the pool's refs in order (4 bytes a page, 16384 pages a step), which
// makes "the lowest free page first" a prefix sum and every result independent
// of the order in which threads run.  Only sums into refs are atomic, and
// those commute.  The copies are bound by HBM.
#include "paged.h"
#include "spec_common.cuh"

namespace spec {

constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kPerThread = 16;  // pages of a thread in a step
constexpr int kForkThreads = 256;

__host__ __device__ __forceinline__ long long pages_for(long long tokens, int page_log2)
{
    return (tokens + (1ll << page_log2) - 1) >> page_log2;
}
__device__ __forceinline__ bool in_pool(const PagesArgs &p, int page) { return page >= 0 && page < p.P; }

size_t page_workspace(int B, int MP, int P)
{
    const size_t fork = (size_t)B * ((size_t)MP + 1), reserve = 5 * (size_t)B + (size_t)P, compact = 3 * (size_t)P + 1;
    const size_t most = fork > reserve ? fork : reserve;
    return align256((most > compact ? most : compact) * 4);
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// Every sequence reads its source's row as it was before the call, so the new
// rows wait in the workspace ([B, MP], then [B] pages or -1: refused) until all
// have been read.
__global__ void __launch_bounds__(kForkThreads) fork_read_kernel(const ForkArgs a)
{
    const PagesArgs &p = a.p;
    const int b = blockIdx.x, t = threadIdx.x;
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
        for (int i = t; i < n; i += kForkThreads)
            ok &= in_pool(p, p.table[(size_t)src * p.MP + i]);
        for (int i = t; i < had; i += kForkThreads)
            ok &= in_pool(p, p.table[(size_t)dst * p.MP + i]);
    }
    ok = __syncthreads_and(ok);
    if (t == 0) {
        p.ws[(size_t)p.B * p.MP + b] = ok ? n : -1;
        if (p.flags)
            p.flags[b] = ok ? 0u : SPEC_FLAG_BAD_STATE;
    }
    if (!ok)
        return;
    for (int i = t; i < p.MP; i += kForkThreads) {
        const int page = i < n ? p.table[(size_t)src * p.MP + i] : -1;
        p.ws[(size_t)b * p.MP + i] = page;
        if (i < n)
            atomicAdd(p.refs + page, 1);
        if (i < had)
            atomicSub(p.refs + p.table[(size_t)dst * p.MP + i], 1);
    }
}

__global__ void __launch_bounds__(kForkThreads) fork_write_kernel(const ForkArgs a)
{
    const PagesArgs &p = a.p;
    const int b = blockIdx.x, n = p.ws[(size_t)p.B * p.MP + b];
    if (n < 0)
        return;
    const int dst = a.dst ? a.dst[b] : b;
    for (int i = threadIdx.x; i < p.MP; i += kForkThreads)
        p.table[(size_t)dst * p.MP + i] = p.ws[(size_t)b * p.MP + i];
    if (threadIdx.x == 0)
        p.held[dst] = n;
}

cudaError_t launch_page_fork(const ForkArgs &a, cudaStream_t st)
{
    fork_read_kernel<<<a.p.B, kForkThreads, 0, st>>>(a);
    fork_write_kernel<<<a.p.B, kForkThreads, 0, st>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// walking the pool in order
// ---------------------------------------------------------------------------
// exclusive prefix of v over the block and its total; `s`: a word per warp.
// Every thread calls; barriers on both sides.
__device__ __forceinline__ int block_before(int v, int *s, int *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, x, m);
        if (lane >= m)
            x += o;
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
            y += o;
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
// What a sequence wants: pages lo .. hi - 1 of its own are written, it ends
// with n pages and had h.
struct Wish {
    int row, lo, hi, n, h;
    bool ok;
};
__device__ __forceinline__ Wish wish_of(const ReserveArgs &a, int b)
{
    const PagesArgs &p = a.p;
    Wish w{};
    w.row = a.idx ? a.idx[b] : b;
    const long long first = a.first[b], total = a.total[b], n = pages_for(total, p.page_log2);
    w.ok = w.row >= 0 && w.row < p.N && first >= 0 && total >= 0 && n <= p.MP;
    if (!w.ok)
        return w;
    w.h = p.held[w.row];
    w.ok = w.h >= 0 && w.h <= p.MP;
    w.n = (int)n;
    const int keep = w.h < w.n ? w.h : w.n;
    w.lo = first < total ? (int)(first >> p.page_log2) : keep;
    w.lo = w.lo < keep ? w.lo : keep;
    w.hi = keep;
    return w;
}

// An entry that will be replaced holds ~page until it is.
__device__ __forceinline__ int entry(const PagesArgs &p, int row, int i)
{
    const int e = __ldcg(p.table + (size_t)row * p.MP + i);
    return e < 0 ? ~e : e;
}

__global__ void __launch_bounds__(kBookThreads) reserve_kernel(const ReserveArgs a)
{
    __shared__ int s_words[32];
    const PagesArgs &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *s_ok = p.ws, *lo = p.ws + p.B, *hi = lo + p.B, *rows = hi + p.B, *want = rows + p.B, *grant = want + p.B;

    // check, and let go of pages behind the new end
    for (int b = warp; b < p.B; b += kBookWarps) {
        const Wish w = wish_of(a, b);
        bool ok = w.ok;
        const bool twice = repeated_row(a.idx, p.B, w.row);
        ok = ok && !twice;
        if (ok)
            for (int i = w.lo + lane; i < w.h; i += 32)
                ok &= in_pool(p, p.table[(size_t)w.row * p.MP + i]);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok)
            for (int i = w.n + lane; i < w.h; i += 32) {
                int32_t *e = p.table + (size_t)w.row * p.MP + i;
                atomicSub(p.refs + *e, 1);
                *e = -1;
            }
        if (lane == 0) {
            s_ok[b] = ok;
            lo[b] = w.lo;
            hi[b] = ok ? w.hi : w.lo;
            rows[b] = w.row;
            if (p.flags)
                p.flags[b] = ok ? 0u : SPEC_FLAG_BAD_STATE;
            if (a.copies) {
                a.copies[2 * b] = -1;
                a.copies[2 * b + 1] = -1;
            }
        }
    }
    __threadfence();
    __syncthreads();

    // Of the sequences that will write a shared page each takes another, but
    // the last of them where nobody else names it.  A page is shared at the
    // same place of every table that names it (fork copies rows).
    for (int b = warp; b < p.B; b += kBookWarps) {
        int swaps = 0;
        for (int c = lo[b]; c < hi[b]; c += 32) {
            const int i = c + lane;
            const int page = i < hi[b] ? entry(p, rows[b], i) : 0;
            const int refs = i < hi[b] ? __ldcg(p.refs + page) : 0;
            unsigned shared = __ballot_sync(0xFFFFFFFFu, refs > 1);
            while (shared) {
                const int l = __ffs(shared) - 1, at = c + l;
                shared &= shared - 1;
                const int which = __shfl_sync(0xFFFFFFFFu, page, l);
                int before = 0;
                for (int o = lane; o < b; o += 32)
                    before += lo[o] <= at && at < hi[o] && entry(p, rows[o], at) == which;
                before = __reduce_add_sync(0xFFFFFFFFu, before);
                if (before < __shfl_sync(0xFFFFFFFFu, refs, l) - 1) {
                    if (lane == 0)
                        __stcg(p.table + (size_t)rows[b] * p.MP + at, ~which);
                    ++swaps;
                }
            }
        }
        if (lane == 0) {
            const Wish w = wish_of(a, b);
            want[b] = s_ok[b] ? swaps + max(0, w.n - w.h) : 0;
        }
    }
    __threadfence();
    __syncthreads();

    // places of the sequences' wishes, in order
    int total = 0;
    for (int c = 0; c < p.B; c += kBookThreads) {
        const int b = c + tid, v = b < p.B ? want[b] : 0;
        int sum;
        const int before = block_before(v, s_words, &sum);
        if (b < p.B)
            want[b] = total + before;
        total += sum;
        if (total > p.P)
            total = p.P + 1;  // more than there can be: enough to know
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
    if (tid == 0 && a.missing)
        *a.missing = enough ? 0 : total - found;
    __threadfence();
    __syncthreads();

    for (int b = warp; b < p.B; b += kBookWarps) {
        if (!s_ok[b])
            continue;
        const Wish w = wish_of(a, b);
        int at = want[b];
        for (int c = w.lo; c < w.n; c += 32) {
            const int i = c + lane;
            int32_t *e = p.table + (size_t)w.row * p.MP + (i < w.n ? i : 0);
            const int old = i < w.hi ? *e : 0;
            const bool fresh = i < w.n && (i < w.hi ? old < 0 : enough);
            const unsigned all = __ballot_sync(0xFFFFFFFFu, fresh && enough);
            if (fresh && !enough)
                *e = ~old;  // as it was
            if (fresh && enough) {
                const int page = grant[at + __popc(all & ((1u << lane) - 1))];
                *e = page;
                p.refs[page] = 1;
                if (i < w.hi) {
                    atomicSub(p.refs + ~old, 1);
                    const int first = a.first[b];
                    if (a.copies && i == first >> p.page_log2 && (first & ((1 << p.page_log2) - 1))) {
                        a.copies[2 * b] = ~old;
                        a.copies[2 * b + 1] = page;
                    }
                }
            }
            at += __popc(all);
        }
        if (lane == 0)
            p.held[w.row] = enough ? w.n : w.hi;
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
    __threadfence();
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
}

__global__ void __launch_bounds__(kForkThreads) rename_kernel(const CompactArgs a)
{
    const PagesArgs &p = a.p;
    const int *place = p.ws + 2 * (size_t)p.P;
    const int live = place[p.P], row = blockIdx.x, n = min(p.held[row], p.MP);
    for (int i = threadIdx.x; i < n; i += kForkThreads) {
        int32_t *e = p.table + (size_t)row * p.MP + i;
        if (*e >= live && *e < p.P)
            *e = place[*e];
    }
}

cudaError_t launch_page_compact(const CompactArgs &a, cudaStream_t st)
{
    compact_kernel<<<1, kBookThreads, 0, st>>>(a);
    if (a.p.N > 0)
        rename_kernel<<<a.p.N, kForkThreads, 0, st>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 4;  // 16-byte words of a thread in flight
constexpr int kCopyChunk = kCopyThreads * kCopyEach * 16;

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PageCopyArgs a)
{
    const int n = a.n_pairs ? max(0, min(*a.n_pairs, a.M)) : a.M;
    if (blockIdx.x == 0 && a.err) {
        int bad = 0;
        for (int c = 0; c < n; c += kCopyThreads) {
            const int i = c + threadIdx.x;
            const int from = i < n ? a.pairs[2 * i] : -1, to = i < n ? a.pairs[2 * i + 1] : -1;
            bad += __syncthreads_count(from != -1 && (from < 0 || from >= a.P || to < 0 || to >= a.P));
        }
        if (threadIdx.x == 0)
            *a.err = bad;
    }
    const int chunks = (int)((a.bytes + kCopyChunk - 1) / kCopyChunk);
    const long long items = (long long)n * a.slabs * chunks;
    for (long long w = blockIdx.x; w < items; w += gridDim.x) {
        const int i = (int)(w / ((long long)a.slabs * chunks));
        const int rest = (int)(w - (long long)i * a.slabs * chunks), slab = rest / chunks, chunk = rest - slab * chunks;
        const int from = a.pairs[2 * i], to = a.pairs[2 * i + 1];
        if (from < 0 || from >= a.P || to < 0 || to >= a.P)
            continue;
        unsigned char *base = a.pool + (long long)slab * a.P * a.bytes;
        const long long off = (long long)chunk * kCopyChunk;
        const uint4 *src = reinterpret_cast<const uint4 *>(base + from * a.bytes + off);
        uint4 *dst = reinterpret_cast<uint4 *>(base + to * a.bytes + off);
        const int words = (int)(min((long long)kCopyChunk, a.bytes - off) / 16);
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
    const long long items = (long long)a.M * a.slabs * ((a.bytes + kCopyChunk - 1) / kCopyChunk);
    const long long most = 152 * 8;
    page_copy_kernel<<<(unsigned)(items < 1 ? 1 : items < most ? items : most), kCopyThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace spec
