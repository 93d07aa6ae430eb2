// attend_common.cuh -- how attention's work is split over CTAs and joined
// again, shared by its kernels (attend_simt.cu, attend_few.cu, attend_tc.cu; over pages
// attend_q4.cu, attend_q4_tc.cu).
//
// A unit is (sequence, key head, group of query rows); its keys are cut into
// tiles.  The query rows of a key head are packed token-major: row r is token
// r / G, query head h * G + r % G, so the G heads that share a key head read
// its keys once.  A round's tiles are those of the cached prefix and one for
// the nodes; the tiles of all units, laid end to end, are dealt out in equal
// contiguous runs to the CTAs.  Every CTA finds its run by itself from the
// lengths on the device, so no host value and no extra launch is needed, and
// a ragged batch is as balanced as a uniform one.  A unit cut by a run's end
// leaves its parts (unnormalised sums, running maximum, weight sum) in the
// workspace; the last CTA to arrive joins them in part order, so results do
// not depend on which that was.
#pragma once

#include "forward.h"
#include "spec_common.cuh"

namespace spec {

constexpr int kAttendCtas = kSms;  // CTAs of a round's launch: one per SM
constexpr int kMinTiles = 2;      // smallest run worth a CTA of its own

struct AttendUnit {
    int b, h;
    int row0, n_rows;      // first query row of the unit within its sequence, and how many
    Seq seq;
    int tile, tile_end;    // this CTA's tiles of the unit
    int n_tiles;           // tiles of the unit
    int seen_first, seen_last;  // prompt: keys that the first and the last query row see
    int part, n_parts;     // place among the unit's parts
    int first_cta;         // CTA that has part 0
};

// tiles of one sequence's unit, and units of the sequence per key head.  IDLE: tiles
// that a unit's start and end cost, counted behind its own; known to the compiler, so
// that a walk without any is none the longer for it (as a number of the call it cost
// the kernels over a 16-bit cache registers: attend_simt<bf16, 4, 2> spilt 816 / 704
// bytes in place of 692 / 692, attend_simt<half, 4, 4> 120 / 148 in place of 80 / 84).
template <int IDLE>
struct UnitShape {
    int tile_keys;  // keys of a tile
    int unit_rows;  // query rows of a unit
    int G;          // query rows of a token
    static constexpr int idle = IDLE;
};
using Shape = UnitShape<0>;
static_assert(sizeof(Shape) == 3 * sizeof(int), "nothing to carry along for units that idle for nothing");
template <typename SH>
__device__ __forceinline__ int round_tiles(const Seq &s, const SH &sh)
{
    return (s.prefix + sh.tile_keys - 1) / sh.tile_keys + 1;
}
template <typename SH>
__device__ __forceinline__ int unit_groups(const Seq &s, const SH &sh)
{
    return (int)(((uint32_t)s.n * sh.G + sh.unit_rows - 1) / (uint32_t)sh.unit_rows);
}
// tiles of a sequence; over all sequences they are fewer than 2^31 (checked on
// the host), so that the walk needs no 64-bit division
template <typename SH>
__device__ __forceinline__ uint32_t round_weight(const Seq &s, const SH &sh, int H)
{
    return (uint32_t)H * unit_groups(s, sh) * (round_tiles(s, sh) + SH::idle);
}

// The run of this CTA: filled by the whole CTA, read by every role.
struct Run {
    uint32_t begin, end;   // tiles, over all sequences
    uint32_t per;          // tiles of a full run
    uint32_t seq_begin;    // first tile of sequence b
    int b;                 // sequence that holds `begin`
};

// Exclusive prefix of v over the block; total in *total.  s: one value per warp.
template <int THREADS>
__device__ uint32_t block_exclusive(uint32_t v, uint32_t *s, uint32_t *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, x, m);
        if (lane >= m)
            x += o;
    }
    if (lane == 31)
        s[w] = x;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < w)
            before += s[i];
        sum += s[i];
    }
    *total = sum;
    return before + x - v;
}

// ---------------------------------------------------------------------------
// waits that gave up
// ---------------------------------------------------------------------------
constexpr size_t kPartHead = SPEC_ATTEND_ZERO;
// the head's last word: not 0 once a wait of a call on the workspace gave up
constexpr int kGaveUpWord = kPartHead / sizeof(int) - 1;
static_assert(2 * kAttendCtas <= kGaveUpWord, "one counter per CTA");
// A CTA that gives up leaves the rest of its run undone, and parts of cut units
// uncounted, so that the counters say nothing any more: SPEC_FLAG_TIMEOUT is
// the whole call's, and every later round's on the workspace until its head is
// cleared.  (A prompt call's flags are written by its first CTA as it starts,
// seconds before any wait can run out.)
__device__ __forceinline__ bool gave_up(const AttendArgs &a)
{
    return *reinterpret_cast<const volatile int *>(static_cast<const int *>(a.ws) + kGaveUpWord) != 0;
}
// by one whole warp, as are the next two
__device__ __forceinline__ void flag_timeout(const AttendArgs &a)
{
    if (a.flags)
#pragma unroll 1
        for (int b = threadIdx.x & 31; b < a.seq.B; b += 32)
            atomicOr(a.flags + b, SPEC_FLAG_TIMEOUT);
}
// by a CTA that gave up
__device__ __forceinline__ void give_up(const AttendArgs &a)
{
    if (a.ws && (threadIdx.x & 31) == 0)
        atomicExch(static_cast<int *>(a.ws) + kGaveUpWord, 1);
    __syncwarp();
    __threadfence();
    flag_timeout(a);
}
// By CTA 0 of a round after it wrote the flags (and a barrier of its threads).
// Either this sees the word of a CTA that gave up, or that CTA's flags come
// after those written here.
__device__ __forceinline__ void flag_if_gave_up(const AttendArgs &a)
{
    __threadfence();
    if (gave_up(a))
        flag_timeout(a);
}

// Every thread takes a contiguous range of sequences; s_run is complete after
// the caller's next __syncthreads.  CTA 0 writes the flags (FLAGS).
template <int THREADS, bool FLAGS = true, typename SH>
__device__ void find_run(const AttendArgs &a, const SH &sh, uint32_t *s_scan, Run *s_run)
{
    const int per_thread = (a.seq.B + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * per_thread, b1 = min(a.seq.B, b0 + per_thread);
    const uint32_t off = FLAGS && blockIdx.x == 0 && gave_up(a) ? SPEC_FLAG_TIMEOUT : 0u;  // a call before this one
    uint32_t w = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(a.seq, a.cache.N, a.cache.S, b);
        w += round_weight(s, sh, a.cache.H);
        if (FLAGS && blockIdx.x == 0 && a.flags)
            a.flags[b] = (s.ok ? 0u : SPEC_FLAG_BAD_STATE) | off;
    }
    uint32_t total;
    uint32_t at = block_exclusive<THREADS>(w, s_scan, &total);
    const uint32_t even = (total + gridDim.x - 1) / gridDim.x;
    const uint32_t per = even < kMinTiles ? kMinTiles : even;
    const uint32_t begin = min(per * blockIdx.x, total);
    if (threadIdx.x == 0) {
        s_run->per = per;
        s_run->begin = begin;
        s_run->end = min(begin + per, total);
    }
    if (at <= begin && begin < at + w) {  // one thread holds it
        if (b1 - b0 > 1)
            for (int b = b0; b < b1; ++b) {
                const uint32_t wb = round_weight(load_seq(a.seq, a.cache.N, a.cache.S, b), sh, a.cache.H);
                if (begin < at + wb) {
                    s_run->b = b;
                    break;
                }
                at += wb;
            }
        else
            s_run->b = b0;
        s_run->seq_begin = at;
    }
}

// The units of a run, in order; each role of a CTA walks its own copy.
template <typename SH = Shape>
struct UnitWalk {
    const AttendArgs *a;
    SH sh;
    Run run;
    uint32_t pos, weight;
    int loaded;  // sequence held in `cur`, or -1
    Seq cur;
    __device__ UnitWalk(const AttendArgs &args, const SH &shape, const Run &r)
        : a(&args), sh(shape), run(r), pos(r.begin), weight(0), loaded(-1)
    {
    }
    __device__ bool next(AttendUnit &u)
    {
        uint32_t tiles, groups, which, t0;
        while (true) {
            if (pos >= run.end)
                return false;
            while (true) {
                if (loaded != run.b) {
                    cur = load_seq(a->seq, a->cache.N, a->cache.S, run.b);
                    weight = round_weight(cur, sh, a->cache.H);
                    loaded = run.b;
                }
                if (pos < run.seq_begin + weight)
                    break;
                run.seq_begin += weight;
                ++run.b;  // ends: run.end is at most the tiles of all sequences
            }
            tiles = round_tiles(cur, sh), groups = unit_groups(cur, sh);
            const uint32_t off = pos - run.seq_begin, span = tiles + SH::idle;
            which = off / span, t0 = off - which * span;
            if (SH::idle == 0 || t0 < tiles)
                break;
            pos += span - t0;  // a run that begins behind a unit's last tile
        }
        const uint32_t left = run.end - pos;
        u.b = run.b;
        u.h = groups == 1 ? which : which / groups;
        u.row0 = (which - u.h * groups) * sh.unit_rows;
        u.n_rows = min(sh.unit_rows, cur.n * sh.G - u.row0);
        u.seq = cur;
        u.tile = t0;
        u.tile_end = t0 + min(tiles - t0, left);
        u.n_tiles = tiles;
        const uint32_t g0 = pos - t0;  // the unit's first tile
        if (t0 == 0 && u.tile_end == (int)tiles) {
            u.first_cta = blockIdx.x;
            u.n_parts = 1;
            u.part = 0;
        } else {
            const uint32_t first = g0 / run.per, last = (g0 + tiles - 1) / run.per;
            u.first_cta = first;
            u.n_parts = last - first + 1;
            u.part = blockIdx.x - first;
        }
        pos += u.tile_end - t0;
        if (SH::idle != 0 && u.tile_end == (int)tiles)
            pos += SH::idle;
        return true;
    }
};

// ---------------------------------------------------------------------------
// parts in the workspace
// ---------------------------------------------------------------------------
// [head: counters, one per CTA, zero between calls] [slots: two per CTA, one for the
// unit that it finishes for others or passes on, one for the unit that starts
// in it and is cut]; a slot is the sums, four columns of all ROWS rows after
// another (threads that hold a row each then write and read side by side), ROWS
// maxima (base 2) and ROWS sums of weights.
__host__ __device__ inline int part_cols(int D) { return (D + 3) & ~3; }
template <int ROWS>
__host__ __device__ inline size_t part_floats(int D)
{
    return (size_t)ROWS * part_cols(D) + 2 * ROWS;
}
template <int ROWS>
__device__ __forceinline__ float *part_slot(const AttendArgs &a, int cta, int part)
{
    float *slots = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kPartHead);
    return slots + (size_t)(2 * cta + (part == 0 ? 1 : 0)) * part_floats<ROWS>(a.cache.D);
}
// place of columns 4 q .. 4 q + 3 of a row in a slot, in floats
template <int ROWS>
__device__ __forceinline__ size_t part_quad(int q, int row)
{
    return ((size_t)q * ROWS + row) * 4;
}
__device__ __forceinline__ int *part_counter(const AttendArgs &a, int cta)
{
    return static_cast<int *>(a.ws) + cta;
}

// place of row r of a unit in q and out, in elements
__device__ __forceinline__ long long row_place(const AttendArgs &a, const AttendUnit &u, int r)
{
    const int t = (u.row0 + r) / a.G, g = u.row0 + r - t * a.G;
    return ((u.seq.tok0 + t) * a.Hq + (long long)u.h * a.G + g) * a.cache.D;
}

template <typename T>
__device__ __forceinline__ T round_to(float x);
template <>
__device__ __forceinline__ float round_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half round_to<__half>(float x) { return __float2half_rn(x); }

// inclusive sums over the warp's lanes
__device__ __forceinline__ uint32_t warp_sums(uint32_t x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, x, m);
        if (lane >= m)
            x += o;
    }
    return x;
}

// The CTA that covers prompt unit blockIdx.x of key head blockIdx.y: units are
// numbered from the last sequence's last rows down, so that the longest of a
// sequence start first.  Every warp finds it from cu: each lane adds up the
// units of B / 32 sequences, whose loads need not wait for one another, then
// the warp goes over those of the lane that has it (against 32 sequences at a
// time: 2000 prompts of 40 tokens 1235 us, 1814; 256 of 60 176, 225).  False:
// no such unit.
__device__ inline bool prompt_unit(const AttendArgs &a, const Shape &sh, AttendUnit &u)
{
    const int lane = threadIdx.x & 31, B = a.seq.B, share = (B + 31) / 32;
    // units of the j-th sequence from the end; those of a call are fewer than 2^31
    auto units = [&](int j) { return (uint32_t)unit_groups(load_seq(a.seq, a.cache.N, a.cache.S, B - 1 - j), sh); };
    uint32_t left = blockIdx.x, mine = 0;
    bool bad = false;
    const int j0 = lane * share, j1 = min(B, j0 + share);
#pragma unroll 4
    for (int j = j0; j < j1; ++j) {
        mine += units(j);
        bad |= a.seq.cu[B - j] < a.seq.cu[B - 1 - j];
    }
    const bool broken = __any_sync(0xFFFFFFFFu, bad);
    int b = -1, which = 0;
    const uint32_t upto = warp_sums(mine);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, left < upto);
    if (hit) {
        const int l = __ffs(hit) - 1;
        if (share == 1) {
            b = B - 1 - l;
            which = (int)(__shfl_sync(0xFFFFFFFFu, upto, l) - 1 - left);  // last group first
        } else {
            left -= __shfl_sync(0xFFFFFFFFu, upto - mine, l);
            for (int c = 0; c < share && b < 0; c += 32) {
                const int j = l * share + c + lane;
                const uint32_t x = warp_sums(c + lane < share && j < B ? units(j) : 0);
                const unsigned in = __ballot_sync(0xFFFFFFFFu, left < x);
                if (in) {
                    const int k = __ffs(in) - 1;
                    b = B - 1 - (l * share + c + k);
                    which = (int)(__shfl_sync(0xFFFFFFFFu, x, k) - 1 - left);
                }
                left -= __shfl_sync(0xFFFFFFFFu, x, 31);
            }
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && a.flags)
        for (int i = threadIdx.x; i < a.seq.B; i += blockDim.x)
            a.flags[i] = !broken && load_seq(a.seq, a.cache.N, a.cache.S, i).ok ? 0u : SPEC_FLAG_BAD_STATE;
    if (b < 0 || broken)
        return false;
    u.b = b;
    u.h = blockIdx.y;
    u.seq = load_seq(a.seq, a.cache.N, a.cache.S, b);
    u.row0 = which * sh.unit_rows;
    u.n_rows = min(sh.unit_rows, u.seq.n * sh.G - u.row0);
    u.seen_first = u.seq.prefix + u.row0 / sh.G + 1;
    u.seen_last = u.seq.prefix + (u.row0 + u.n_rows - 1) / sh.G + 1;
    u.tile = 0;
    u.n_tiles = u.tile_end = (u.seen_last + sh.tile_keys - 1) / sh.tile_keys;
    u.part = u.first_cta = 0;
    u.n_parts = 1;
    return true;
}

// Joins up to P parts of a unit: a thread takes I times 4 Q columns of a row at
// once, and everything that those need comes in one round of loads.
template <typename T, int ROWS, int P, int I, int Q>
__device__ __forceinline__ void join_few_parts(const AttendArgs &a, const AttendUnit &u, int t, int threads)
{
    const int D = a.cache.D, dp = part_cols(D), quads = dp / 4, items = u.n_rows * ((quads + Q - 1) / Q);
    T *out = reinterpret_cast<T *>(a.out);
    const bool wide = D % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    for (int w0 = t; w0 < items; w0 += I * threads) {
        float mp[I][P], lp[I][P];
        float4 x[I][P][Q];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int w = w0 + i * threads, g = w / u.n_rows, r = w - g * u.n_rows;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const bool in = w < items && p < u.n_parts;
                const float *slot = part_slot<ROWS>(a, u.first_cta + p, p);
                mp[i][p] = in ? __ldcg(slot + (size_t)ROWS * dp + r) : -INFINITY;
                lp[i][p] = in ? __ldcg(slot + (size_t)ROWS * dp + ROWS + r) : 0.0f;
#pragma unroll
                for (int k = 0; k < Q; ++k)
                    x[i][p][k] = in && Q * g + k < quads
                                     ? __ldcg(reinterpret_cast<const float4 *>(slot + part_quad<ROWS>(Q * g + k, r)))
                                     : make_float4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int w = w0 + i * threads, g = w / u.n_rows, r = w - g * u.n_rows;
            if (w >= items)
                break;
            float m = -INFINITY, l = 0.0f, o[4 * Q] = {};
#pragma unroll
            for (int p = 0; p < P; ++p)
                m = fmaxf(m, mp[i][p]);
            const float m0 = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const float f = exp2f(mp[i][p] - m0);
                l = fmaf(f, lp[i][p], l);
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    o[4 * k] = fmaf(f, x[i][p][k].x, o[4 * k]);
                    o[4 * k + 1] = fmaf(f, x[i][p][k].y, o[4 * k + 1]);
                    o[4 * k + 2] = fmaf(f, x[i][p][k].z, o[4 * k + 2]);
                    o[4 * k + 3] = fmaf(f, x[i][p][k].w, o[4 * k + 3]);
                }
            }
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            T *dst = out + row_place(a, u, r) + 4 * Q * g;
            T v[4 * Q];
#pragma unroll
            for (int e = 0; e < 4 * Q; ++e)
                v[e] = round_to<T>(o[e] * inv);
#pragma unroll
            for (int e = 0; e < 4 * Q; e += 8) {
                if (4 * Q * g + e >= D)
                    break;
                if (wide) {
#pragma unroll
                    for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
                        uint4 y;
                        memcpy(&y, v + e + 16 / sizeof(T) * k, 16);
                        reinterpret_cast<uint4 *>(dst + e)[k] = y;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (4 * Q * g + e + k < D)
                            dst[e + k] = v[e + k];
                }
            }
        }
    }
}

// Joins a unit's parts: O = sum 2^(m_p - m) O_p / sum 2^(m_p - m) l_p.  Called
// by all `threads` threads of which this is t, after every part was seen;
// `sync` is a barrier among them that orders their writes to the workspace
// (false: it gave up).  What a join costs is its rounds of loads, a latency
// each: with few parts everything comes in one (join_few_parts; decoding at
// batch 32 43 -> 40 us, trees of 64 nodes and 7 heads 119 -> 115).  Else every
// row's factors are formed first where a thread has many rows to join, in
// place of the parts' maxima, or come with the sums where it has few.  A row
// that no part saw anything for (every l zero) gives zeros.
template <typename T, int ROWS, typename Sync>
__device__ bool join_parts(const AttendArgs &a, const AttendUnit &u, int t, int threads, Sync sync)
{
    const int D = a.cache.D, dp = part_cols(D), quads = dp / 4, groups = (quads + 3) / 4;
    T *out = reinterpret_cast<T *>(a.out);
    auto stats = [&](int p) { return part_slot<ROWS>(a, u.first_cta + p, p) + (size_t)ROWS * dp; };
    // a row's maximum and the inverse of its sum
    auto whole_row = [&](int r, float &m0, float &inv) {
        float m = -INFINITY;
#pragma unroll 4
        for (int p = 0; p < u.n_parts; ++p)
            m = fmaxf(m, __ldcg(stats(p) + r));
        m0 = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
#pragma unroll 4
        for (int p = 0; p < u.n_parts; ++p)
            l = fmaf(exp2f(__ldcg(stats(p) + r) - m0), __ldcg(stats(p) + ROWS + r), l);
        inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    };
    const bool many = u.n_rows * groups > 4 * threads;
    if (!many && u.n_parts <= 4) {
        join_few_parts<T, ROWS, 4, 1, 2>(a, u, t, threads);
        return true;
    }
    if (many && u.n_parts == 2) {
        join_few_parts<T, ROWS, 2, 2, 4>(a, u, t, threads);
        return true;
    }
    if (many) {
        for (int r = t; r < u.n_rows; r += threads) {
            float m0, inv;
            whole_row(r, m0, inv);
#pragma unroll 4
            for (int p = 0; p < u.n_parts; ++p)
                __stcg(stats(p) + r, exp2f(__ldcg(stats(p) + r) - m0) * inv);
        }
        if (!sync())
            return false;
    }
    for (int i = t; i < u.n_rows * groups; i += threads) {
        const int g = i / u.n_rows, r = i - g * u.n_rows, q0 = 4 * g;
        float o[16] = {}, m0 = 0.0f, inv = 1.0f;
        if (!many)
            whole_row(r, m0, inv);
        // parts a round of loads: four where the caller has the registers (18 nodes
        // of 7 heads, 8 sequences: 55 -> 47 us; small units 41 -> 45)
        constexpr int NB = ROWS >= 128 ? 4 : 2;
        for (int p0 = 0; p0 < u.n_parts; p0 += NB) {
            float f[NB];
            float4 x[NB][4];
#pragma unroll
            for (int p = 0; p < NB; ++p) {
                const bool in = p0 + p < u.n_parts;
                const float *slot = part_slot<ROWS>(a, u.first_cta + p0 + p, p0 + p);
                f[p] = in ? __ldcg(slot + (size_t)ROWS * dp + r) : (many ? 0.0f : -INFINITY);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[p][k] = in && q0 + k < quads
                                  ? __ldcg(reinterpret_cast<const float4 *>(slot + part_quad<ROWS>(q0 + k, r)))
                                  : make_float4(0, 0, 0, 0);
            }
#pragma unroll
            for (int p = 0; p < NB; ++p) {
                const float w = many ? f[p] : exp2f(f[p] - m0) * inv;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o[4 * k] = fmaf(w, x[p][k].x, o[4 * k]);
                    o[4 * k + 1] = fmaf(w, x[p][k].y, o[4 * k + 1]);
                    o[4 * k + 2] = fmaf(w, x[p][k].z, o[4 * k + 2]);
                    o[4 * k + 3] = fmaf(w, x[p][k].w, o[4 * k + 3]);
                }
            }
        }
        T *dst = out + row_place(a, u, r) + 16 * g;
        if (D % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0) {
            T v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
                v[e] = round_to<T>(o[e]);
            constexpr int N = sizeof(T);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                uint4 y;
                memcpy(&y, v + 16 / N * k, 16);
                reinterpret_cast<uint4 *>(dst)[k] = y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (16 * g + e < D)
                    dst[e] = round_to<T>(o[e]);
        }
    }
    return true;
}

}  // namespace spec
