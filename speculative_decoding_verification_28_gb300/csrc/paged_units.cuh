// paged_units.cuh -- the walk over a CTA's units for the attention kernels over
// pages: one warp walks and hands the units to the others through a ring in
// shared memory.  (Walked by every role for itself, as in the kernels over a
// contiguous cache, a unit costs each role some 600 instructions that nothing
// keeps in the instruction cache: 20000 clocks a unit, against 5000 a tile.)
#pragma once

#include "attend_common.cuh"
#include "paged.h"
#include "q4.cuh"
#include "tcgen.cuh"

namespace spec {

constexpr int kUnitRing = 4;

struct PagedUnit {
    int b, h, row0, n_rows;      // query rows row0 .. of key head h; n_rows 0: no more units
    int n, prefix, row;          // nodes, keys in pages, table row
    int tile, tile_end, n_tiles;
    int part, n_parts, first_cta;
    int pad[3];
};
struct PagedRing {
    PagedUnit unit[kUnitRing];
    uint64_t full[kUnitRing], empty[kUnitRing];
};

// by one thread; `readers` warps read every unit
__device__ __forceinline__ void units_init(PagedRing &r, int readers)
{
    for (int i = 0; i < kUnitRing; ++i) {
        mbar_init(&r.full[i], 1);
        mbar_init(&r.empty[i], readers);
    }
}
// The walking warp: puts unit n (null: the end) into the ring.
__device__ __forceinline__ bool units_put(PagedRing &r, uint32_t n, const AttendUnit *u, int *abort, long long limit)
{
    const int i = n % kUnitRing;
    if (!__all_sync(0xFFFFFFFFu, wait_phase(&r.empty[i], ((n / kUnitRing) & 1) ^ 1, abort, limit)))
        return false;
    if ((threadIdx.x & 31) == 0) {
        PagedUnit &p = r.unit[i];
        p.n_rows = 0;
        if (u) {
            p.b = u->b;
            p.h = u->h;
            p.row0 = u->row0;
            p.n_rows = u->n_rows;
            p.n = u->seq.n;
            p.prefix = u->seq.prefix;
            p.row = u->seq.row;
            p.tile = u->tile;
            p.tile_end = u->tile_end;
            p.n_tiles = u->n_tiles;
            p.part = u->part;
            p.n_parts = u->n_parts;
            p.first_cta = u->first_cta;
        }
        mbar_arrive(&r.full[i]);
    }
    __syncwarp();
    return true;
}
// A reading warp: unit n, or false at the end (or after a wait that gave up).
__device__ __forceinline__ bool units_get(PagedRing &r, uint32_t n, PagedUnit &u, int *abort, long long limit)
{
    const int i = n % kUnitRing;
    if (!__all_sync(0xFFFFFFFFu, wait_phase(&r.full[i], (n / kUnitRing) & 1, abort, limit)))
        return false;
    u = r.unit[i];
    return u.n_rows != 0;
}
// The same, where it lies: a unit stays there until units_done.
__device__ __forceinline__ const PagedUnit *units_at(const PagedRing &r, uint32_t n) { return &r.unit[n % kUnitRing]; }
__device__ __forceinline__ bool units_wait(PagedRing &r, uint32_t n, int *abort, long long limit)
{
    return __all_sync(0xFFFFFFFFu, wait_phase(&r.full[n % kUnitRing], (n / kUnitRing) & 1, abort, limit)) &&
           units_at(r, n)->n_rows != 0;
}
// ... which is done with it
__device__ __forceinline__ void units_done(PagedRing &r, uint32_t n)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&r.empty[n % kUnitRing]);
}

// place of row r of a unit in q and out, in elements
__device__ __forceinline__ long long row_place(const AttendArgs &a, const PagedUnit &u, int r)
{
    const int t = (u.row0 + r) / a.G, g = u.row0 + r - t * a.G;
    return (((long long)u.b * a.seq.T + t) * a.Hq + (long long)u.h * a.G + g) * a.cache.D;
}
// nodes that row r of a unit sees
__device__ __forceinline__ uint64_t row_nodes(const AttendArgs &a, const PagedUnit &u, int r)
{
    const int tok = (u.row0 + r) / a.G;
    const uint64_t bits = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
    return u.n < 64 ? bits & ((1ull << u.n) - 1) : bits;
}
// the unit as the joins want it
__device__ __forceinline__ AttendUnit join_unit(const AttendArgs &a, const PagedUnit &p)
{
    AttendUnit u{};
    u.b = p.b;
    u.h = p.h;
    u.row0 = p.row0;
    u.n_rows = p.n_rows;
    u.seq.tok0 = (long long)p.b * a.seq.T;
    u.part = p.part;
    u.n_parts = p.n_parts;
    u.first_cta = p.first_cta;
    return u;
}

// The copies of a tile of KEYS keys of a unit, by the whole walking warp: codes
// and scales of its keys and values, a copy a lane (page of 16: 32 lanes), as K codes,
// V codes, K scales, V scales one after another.  What does not change from tile to tile is
// worked out once a unit: this warp's time a tile is what the others wait for.
template <int D, int KEYS>
struct TileCopies {
    static constexpr int kCodes = KEYS * q4_codes(D), kScales = KEYS * q4_scales(D);
    const int32_t *table, *row;
    const unsigned char *first;  // this lane's part of page 0, of key head 0
    const unsigned char *base;   // ... of the unit's key head
    long long block, page_bytes;
    int MP, P, log2, log2_piece, per;  // a piece: tokens that lie side by side in a page, up to a tile; pieces of a tile
    int width, bytes, to, mine;        // of this lane's part of a piece: a token's bytes, all, place in the tile; its piece
    int prefix, have, held;            // this lane's table entry: that of piece have + lane of the sequence
    __device__ __forceinline__ TileCopies(const AttendQ4Args &x)
    {
        const int which = threadIdx.x & 3;
        table = x.pool.table;
        MP = x.pool.MP;
        P = x.pool.P;
        log2 = x.pool.page_log2;
        log2_piece = min(31 - __clz(KEYS), log2);
        per = KEYS >> log2_piece;
        mine = (threadIdx.x & 31) >> 2;
        block = x.pool.block;
        page_bytes = x.pool.page_bytes;
        width = which < 2 ? q4_codes(D) : q4_scales(D);
        bytes = width << log2_piece;
        to = (which & 1 ? (which < 2 ? kCodes : kScales) : 0) + (which < 2 ? 0 : 2 * kCodes) + mine * bytes;
        first = x.pool.pool + (which & 1 ? x.v_block : x.k_block) * block + (which < 2 ? 0 : (long long)q4_codes(D) << log2);
    }
    __device__ __forceinline__ void begin(const AttendUnit &u)
    {
        row = table + (size_t)u.seq.row * MP;
        base = first + u.h * block;
        prefix = u.seq.prefix;
        have = -1;
    }
    // page of this lane's piece of the tile; UP: whether tiles go up
    template <bool UP>
    __device__ __forceinline__ int page_of(int tile)
    {
        const int p0 = tile * per;
        if (have < 0 || (UP ? p0 + per > have + 32 : p0 < have)) {
            have = UP ? p0 : max(0, p0 + per - 32);
            const int tok = (have + (threadIdx.x & 31)) << log2_piece;  // fewer than 2^31 and a few pages: no overflow
            held = tok >= 0 && tok < prefix ? __ldg(row + (tok >> log2)) : 0;
            held = (unsigned)held < (unsigned)P ? held : 0;  // flagged at the walk's end
        }
        return __shfl_sync(0xFFFFFFFFu, held, p0 - have + (mine < per ? mine : 0));
    }
    __device__ __forceinline__ void issue(int tile, int page, unsigned char *slot, uint64_t *bar) const
    {
        const int valid = min(KEYS, prefix - tile * KEYS), pieces = (valid + (1 << log2_piece) - 1) >> log2_piece;
        if ((threadIdx.x & 31) == 0)
            mbar_arrive_expect_tx(bar, (uint32_t)((pieces << log2_piece) * 2 * (q4_codes(D) + q4_scales(D))));
        __syncwarp();
        if (mine < pieces) {
            const int in_page = (tile * KEYS) & ((1 << log2) - 1);  // not 0 only where a piece is as long as the tile
            bulk_g2s(slot + to, base + page * page_bytes + in_page * width, (uint32_t)bytes, bar);
        }
    }
};

// A unit's queries and nodes on their way to L2, by the walking warp: they
// are read when the unit's turn comes, with nothing else to do meanwhile.
template <typename T, int D>
__device__ __forceinline__ void prefetch_unit(const AttendArgs &a, const AttendUnit &u)
{
    const int lane = threadIdx.x & 31;
    auto fetch = [](const T *p, long long elements) {
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"((uint32_t)(elements * 2)) : "memory");
    };
    const int t0 = u.row0 / a.G, t1 = (u.row0 + u.n_rows - 1) / a.G;
    for (int t = t0 + lane; t <= t1; t += 32)
        fetch(reinterpret_cast<const T *>(a.q) + ((u.seq.tok0 + t) * a.Hq + (long long)u.h * a.G) * D, (long long)a.G * D);
    if (u.tile_end == u.n_tiles && lane < 2)
        fetch(reinterpret_cast<const T *>(a.staged) +
                  ((lane ? a.st_v : a.st_k) + (long long)u.b * a.cache.H + u.h) * a.seq.T * D,
              (long long)u.seq.n * D);
}

// By the walking warp at its end: flags of the sequences whose first tile this
// CTA had, and by CTA 0 of those that have none.
template <typename SH>
__device__ __noinline__ void paged_flags(const AttendQ4Args &x, const SH &sh, const Run &run)
{
    const AttendArgs &a = x.a;
    if (!a.flags)
        return;
    const int lane = threadIdx.x & 31;
    UnitWalk<SH> again(a, sh, run);
    AttendUnit u{};
    while (again.next(u)) {
        if (u.tile != 0 || u.h != 0 || u.row0 != 0)
            continue;
        const int32_t *row = x.pool.table + (size_t)u.seq.row * x.pool.MP;
        const int pages = (int)(((long long)u.seq.prefix + (1 << x.pool.page_log2) - 1) >> x.pool.page_log2);
        bool fine = true;
#pragma unroll 8
        for (int i = lane; i < pages; i += 32)
            fine &= (unsigned)__ldg(row + i) < (unsigned)x.pool.P;
        fine = __all_sync(0xFFFFFFFFu, fine);
        if (lane == 0)
            a.flags[u.b] = fine ? 0u : SPEC_FLAG_BAD_STATE;
    }
    if (blockIdx.x == 0)
        for (int b = lane; b < a.seq.B; b += 32) {
            const Seq q = load_seq(a.seq, a.cache.N, a.cache.S, b);
            if (q.n == 0)
                a.flags[b] = q.ok ? 0u : SPEC_FLAG_BAD_STATE;
        }
    __syncwarp();
    flag_if_gave_up(a);
}

}  // namespace spec
