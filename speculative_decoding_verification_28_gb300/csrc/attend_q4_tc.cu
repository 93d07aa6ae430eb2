// attend_q4_tc.cu -- attention of a round over pages of 4-bit keys and values on
// the fifth-generation tensor cores, for rounds with many query rows a key head
// (chains of shared heads, trees).
//
//   S = Q K^T in TMEM;  P = 2^(c S - m) in TMEM, fp16;  O += P V in TMEM, fp32
//
// as in attend_tc.cu, with up to 128 query rows a unit.  What is different is
// where the operands come from: pages arrive as codes (cp.async.bulk, a ring of
// tiles of 128 keys), and eight warps expand them to fp16 tiles in the
// 128-byte-swizzled form that tcgen05 reads, each 16 bytes of codes (a group, one scale)
// by one thread.  Expanded values are 128 times too small (q4_expand.cuh) and the
// eight dimensions of a word of codes stand in the order 0 4 1 5 2 6 3 7: queries
// follow that order, and O's columns are put back as they are stored.  Queries are the
// first operand of S and lie in TMEM (shared memory is what bounds this kernel):
// fp16, bf16 rows times a power of two; and for the nodes' tile, which is in
// the storage type, as they are.
//
// A part of a unit begins with the nodes, if it has them, so that their O is in
// its own units until the first tile of the prefix, whose pass over O divides it by 128.
//
//   softmax warps   128 threads, one per query row (attend_few.cu's softmax)
//   mma warp        issues S = Q K^T one tile ahead of O += P V, across units
//   load warp       codes and scales of a tile's pages
//   expand warps    tiles of the prefix; the nodes' tile and the queries
#include <type_traits>

#include "paged.h"
#include "q4_expand.cuh"
#include "tcgen.cuh"

namespace spec {

constexpr int kQtRows = 128;
constexpr int kQtExpand = 8;  // warps
constexpr int kQtThreads = 32 * (4 + 4 + kQtExpand);  // whole warpgroups, see below
constexpr int kQtTmemP = 64;  // columns of a score buffer where its weights begin
constexpr uint32_t kQtTmemO = 256, kQtTmemQ = 384;  // and 64 columns of queries in the storage type behind 64 of fp16
constexpr int kQtUnits = 4;   // units whose words may be live at once

template <int D>
struct QtShape {
    static constexpr int kPanels = D / 64;
    static constexpr int kPanel = kKeys * 128;
    static constexpr int kTile = kPanels * kPanel;  // bytes of an expanded tile
    static constexpr int kCodes = kKeys * q4_codes(D), kScales = kKeys * q4_scales(D);
    static constexpr int kStage = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kBuf = 2;  // expanded tiles of keys, and of values
    static constexpr int kSmem = 2 * kBuf * kTile + kStages * kStage + 1024;
};
template <int STAGES>
struct QtShared {
    uint64_t st_full[STAGES], st_empty[STAGES];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done, joined, settled, never;
    uint32_t asked;  // tiles that were copied in all
    uint32_t scan[16];
    Run run;
    uint32_t tmem;
    int abort, last;
    float c[kQtUnits][kQtRows];        // what takes a row's scores to base 2
    int odd[kQtUnits][kQtExpand];      // whether a value of the nodes is not finite
};

// A part's tiles in the order in which they are taken: the last, the nodes', first.
__device__ __forceinline__ Tile qt_tile(const AttendUnit &u, int tile)
{
    Tile t;
    t.nodes = tile == u.n_tiles - 1;
    t.valid = t.nodes ? u.seq.n : min(kKeys, u.seq.prefix - tile * kKeys);
    t.masked = t.nodes;
    return t;
}

// where 16 bytes `chunk` of a row's 128 in a swizzled panel lie
__device__ __forceinline__ int swizzled(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// The values of a tile's keys or values, expanded by one warp of kQtExpand.
template <int D>
__device__ __forceinline__ void qt_expand(const unsigned char *codes, const unsigned char *scales, unsigned char *to,
                                          int warp, int valid)
{
    // four keys' halves of a panel to eight lanes: reads collide twice, writes not at all
    const int lane = threadIdx.x & 31, half = lane & 1, k2 = lane >> 1 & 3;
    constexpr int kIter = D == 128 ? 2 : 1;
    const int panel = D == 128 ? lane >> 3 & 1 : 0;
    const int sub = D == 128 ? lane >> 4 << 2 : lane >> 3 << 2;
    const int group = 2 * panel + half;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int key = warp * (kKeys / kQtExpand) + 8 * i + sub + k2;
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + key * q4_codes(D) + group * 16);
        const uint32_t b = key < valid ? scales[key * q4_scales(D) + group] : 0;
        const Scale2 s(b * 0x00800080u);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
            q4_expand(x[k], s, y);
            *reinterpret_cast<uint4 *>(to + panel * QtShape<D>::kPanel + swizzled(key, 4 * half + k)) =
                make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
}

// The nodes' keys or values, by one warp; true: some value was not finite (and
// is 0 now, CLEAN).
template <typename T, int D, bool CLEAN>
__device__ __forceinline__ bool qt_nodes(const T *rows, unsigned char *to, int warp, int n)
{
    constexpr int kChunks = D / 8;
    const int lane = threadIdx.x & 31, end = (n + 15) & ~15;
    bool odd = false;
    for (int i = warp * 32 + lane; i < end * kChunks; i += 32 * kQtExpand) {
        const int key = i / kChunks, c = i - key * kChunks;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (key < n)
            x = __ldg(reinterpret_cast<const uint4 *>(rows + (size_t)key * D) + c);
        uint32_t y[4];
        pairs_of(x, y);
        if (CLEAN) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((y[k] & TcType<T>::kExp) == TcType<T>::kExp) {
                    y[k] &= 0xFFFF0000u;
                    odd = true;
                }
                if ((y[k] >> 16 & TcType<T>::kExp) == TcType<T>::kExp) {
                    y[k] &= 0x0000FFFFu;
                    odd = true;
                }
            }
        }
        *reinterpret_cast<uint4 *>(to + (c >> 3) * QtShape<D>::kPanel + swizzled(key, c & 7)) =
            make_uint4(y[0], y[1], y[2], y[3]);
    }
    return __any_sync(0xFFFFFFFFu, odd);
}

// A unit's queries to TMEM, a thread a row: fp16 (RAW: as they are).
template <typename T, int D, bool RAW>
__device__ __forceinline__ void qt_queries(const AttendArgs &a, const AttendUnit &u, uint32_t tmem, float *c)
{
    const int row = threadIdx.x & 127;  // TMEM lane
    const uint32_t lanes = (threadIdx.x >> 5 & 3) << 21;
    const bool real = row < u.n_rows;
    const uint4 *p =
        reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.q) + row_place(a, u, real ? row : 0));
    float f = 1.0f;
    int e = 0;
    if constexpr (!RAW && !std::is_same<T, __half>::value) {
        float top = 0.0f;
        if (real)
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                float x[8];
                Storage<T>::unpack(__ldg(p + k), x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = fmaxf(top, fabsf(x[i]));
            }
        e = q4_row_exponent(top);
        f = __uint_as_float((uint32_t)(127 + e) << 23);
    }
    if (!RAW)
        c[row] = a.scale_log2 * exp2f((float)(7 - e));
#pragma unroll 1
    for (int k = 0; k < D / 32; ++k) {
        uint32_t y[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 x = real ? __ldg(p + 4 * k + i) : make_uint4(0, 0, 0, 0);
            if constexpr (RAW || std::is_same<T, __half>::value) {
                pairs_of(x, y + 4 * i);
            } else {
                float v[8];
                Storage<T>::unpack(x, v);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    y[4 * i + d] = TcType<__half>::pack(v[d] * f, v[d + 4] * f);
            }
        }
        tc_st16(tmem + lanes + 16 * k, y);
    }
    tc_wait_st();
    tc_fence_before();
}

// Columns in the order of the expanded words -> as they are.
__device__ __forceinline__ void in_order32(uint32_t *o)
{
#pragma unroll
    for (int w = 0; w < 32; w += 8) {
        const uint32_t x[8] = {o[w], o[w + 2], o[w + 4], o[w + 6], o[w + 1], o[w + 3], o[w + 5], o[w + 7]};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[w + i] = x[i];
    }
}

// Adds what is not finite among the nodes' values to columns col .. col + 31
// of a row that sees it; its weights are positive, so that it stays as it is.
template <typename T, int D>
__device__ __noinline__ void qt_put_back32(const AttendArgs &a, const AttendUnit &u, int tok, int col, uint32_t *o)
{
    const T *values = reinterpret_cast<const T *>(a.staged) + (a.st_v + (long long)u.b * a.cache.H + u.h) * a.seq.T * D;
    const uint64_t bits = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
    for (int key = 0; key < u.seq.n; ++key)
        if (bits >> key & 1)
            for (int e = 0; e < 32; ++e) {
                const float f = Storage<T>::at(values + (size_t)key * D, col + e);
                if (!(fabsf(f) <= 3.4e38f))
                    o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
            }
}

template <typename T, int D>
__global__ void __launch_bounds__(kQtThreads, 1) attend_q4_tc_kernel(const __grid_constant__ AttendQ4Args x)
{
    using Sh = QtShape<D>;
    constexpr int ST = Sh::kStages;
    extern __shared__ unsigned char dyn[];
    __shared__ QtShared<ST> s;
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    unsigned char *keys_p = base, *values_p = base + 2 * Sh::kTile, *stage_p = base + 4 * Sh::kTile;
    const AttendArgs &a = x.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Shape sh{kKeys, kQtRows, a.G};
    constexpr int kMmaWarp = 4, kLoadWarp = 5, kFirstExpand = 8;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&s.st_full[i], 1);
            mbar_init(&s.st_empty[i], kQtExpand);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], kQtExpand);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_full[i], kQtExpand);
            mbar_init(&s.v_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
        }
        mbar_init(&s.q_full, kQtExpand);
        mbar_init(&s.q_empty, 1);
        mbar_init(&s.pv_done, 1);
        mbar_init(&s.joined, 128);
        mbar_init(&s.settled, 1);
        mbar_init(&s.never, 1);
        fence_mbar_init();
        s.abort = 0;
        s.asked = 0;
        s.run.begin = s.run.end = 0;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    __syncthreads();  // run.begin / end above come before find_run's
    find_run<kQtThreads, false>(a, sh, s.scan, &s.run);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;

    // a bounded wait of a whole warp; after one that gave up every role leaves its loop
    const long long limit = a.wait_clocks;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, &s.abort, limit));
    };
    UnitWalk units(a, sh, s.run);
    AttendUnit u{};

    // 512 threads launch with 128 registers each (65536); the softmax keeps 184, the
    // expansion 112, the others 96 (128 * (184 + 2 * 112 + 96) = 64512)
    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        const int log2 = x.pool.page_log2, piece = min(kKeys, 1 << log2), per = kKeys / piece;
        const int which = lane & 3, mine = lane >> 2;  // K codes, V codes, K scales, V scales of one piece of a tile
        const int width = which < 2 ? q4_codes(D) : q4_scales(D);
        const int at_stage = (which & 1 ? (which < 2 ? Sh::kCodes : Sh::kScales) : 0) + (which < 2 ? 0 : 2 * Sh::kCodes);
        const long long first = which & 1 ? x.v_block : x.k_block;
        const long long off = which < 2 ? 0 : (long long)q4_codes(D) << log2;
        uint32_t it = 0;
        bool ok = true;
        while (ok && units.next(u)) {
            const int32_t *row = x.pool.table + (size_t)u.seq.row * x.pool.MP;
            int have = 0x7FFFFFFF, held = 0;  // table entry of piece `have` + lane of the sequence
            for (int tile = min(u.tile_end, u.n_tiles - 1) - 1; ok && tile >= u.tile; --tile, ++it) {
                const int sg = it % ST, valid = min(kKeys, u.seq.prefix - tile * kKeys);
                const int p0 = tile * per;
                if (p0 < have) {
                    have = max(0, p0 + per - 32);
                    const long long tok = (long long)(have + lane) * piece;
                    held = tok < u.seq.prefix ? __ldg(row + (tok >> log2)) : 0;
                    held = held >= 0 && held < x.pool.P ? held : 0;  // flagged below
                }
                const int page = __shfl_sync(0xFFFFFFFFu, held, p0 - have + (mine < per ? mine : 0));
                ok = wait(&s.st_empty[sg], ((it / ST) & 1) ^ 1);
                if (!ok)
                    break;
                const int pieces = (valid + piece - 1) / piece;
                if (lane == 0)
                    mbar_arrive_expect_tx(&s.st_full[sg], (uint32_t)(pieces * piece * 2 * (q4_codes(D) + q4_scales(D))));
                __syncwarp();
                if (mine < pieces) {
                    const unsigned char *blk = x.pool.pool + (first + (long long)page * x.pool.H + u.h) * x.pool.block;
                    const int in_page = (tile * kKeys) & ((1 << log2) - 1);  // of a piece as long as the tile
                    bulk_g2s(stage_p + sg * Sh::kStage + at_stage + mine * piece * width,
                             blk + off + (long long)in_page * width, (uint32_t)(piece * width), &s.st_full[sg]);
                }
            }
        }
        if (lane == 0)
            s.asked = it;
        // flags of the sequences whose first tile this CTA had, and by CTA 0 those that have none
        if (a.flags) {
            UnitWalk again(a, sh, s.run);
            while (again.next(u)) {
                if (u.tile != 0 || u.h != 0 || u.row0 != 0)
                    continue;
                const int32_t *row = x.pool.table + (size_t)u.seq.row * x.pool.MP;
                bool fine = true;
                for (int i = lane; (long long)i << log2 < u.seq.prefix; i += 32) {
                    const int page = __ldg(row + i);
                    fine &= page >= 0 && page < x.pool.P;
                }
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
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------------- mma
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        const uint32_t one = elect_one();
        const uint32_t keys = smem_addr(keys_p), values = smem_addr(values_p);
        auto commit = [&](uint64_t *bar) {
            if (one)
                tc_commit(bar);
        };
        // scores run one tile ahead of weights, across units
        UnitWalk ahead(a, sh, s.run);
        AttendUnit w{};
        bool have = ahead.next(w);
        int wt = w.tile_end - 1;
        uint32_t i = 0, is = 0, nq = 0;  // tiles weighed, tiles scored, units scored
        bool ok = true;
        auto score_next = [&]() {
            const int b = is & 1;
            const Tile tl = qt_tile(w, wt);
            if (wt == w.tile_end - 1)
                ok = ok && wait(&s.q_full, nq & 1);
            ok = ok && wait(&s.k_full[b], (is >> 1) & 1);
            if (!ok)
                return;
            tc_fence_after();
            const int n = min(kKeys, (tl.valid + 15) & ~15);
            const uint32_t ides = tl.nodes ? tc_idesc<T>(n, false) : tc_idesc<__half>(n, false);
            const uint32_t q = tmem + kQtTmemQ + (tl.nodes && !std::is_same<T, __half>::value ? 64 : 0);
            const uint32_t kd = operand(keys + b * Sh::kTile, 16);
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
                mma_ts(one, tmem + b * 128, q + c * 8, kd + (((c / 4) * Sh::kPanel + (c % 4) * 32) >> 4), ides, c > 0);
            commit(&s.s_full[b]);
            commit(&s.k_empty[b]);
            ++is;
            if (--wt < w.tile) {
                commit(&s.q_empty);
                ++nq;
                have = ahead.next(w);
                wt = w.tile_end - 1;
            }
        };
        if (have)
            score_next();
        while (ok && units.next(u)) {
            for (int tile = u.tile_end - 1; ok && tile >= u.tile; --tile) {
                if (have)
                    score_next();
                const int b = i & 1;
                const Tile tl = qt_tile(u, tile);
                ok = ok && wait(&s.p_full[b], (i >> 1) & 1) && wait(&s.v_full[b], (i >> 1) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t ides = tl.nodes ? tc_idesc<T>(D, true) : tc_idesc<__half>(D, true);
                const uint32_t vd = operand(values + b * Sh::kTile, Sh::kPanel), p = tmem + b * 128 + kQtTmemP;
                mma_ts(one, tmem + kQtTmemO, p, vd, ides, tile < u.tile_end - 1);
                for (int c = 1; c < (tl.valid + 15) / 16; ++c)
                    mma_ts(one, tmem + kQtTmemO, p + c * 8, vd + c * (2048 >> 4), ides, 1);
                commit(&s.v_empty[b]);
                commit(&s.pv_done);
                ++i;
            }
        }
    } else if (warp >= kFirstExpand) {
        // ----------------------------------------------------------- expand
        asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        const int e = warp - kFirstExpand;
        uint32_t i = 0, it = 0, n = 0;  // tiles, tiles of the prefix, units
        bool ok = !a.starve || wait(&s.never, 0);
        while (ok && units.next(u)) {
            const bool nodes = u.tile_end == u.n_tiles;
            // keys of the first tile before the queries, which wait for the unit before to be scored
            int odd = 0;
            for (int tile = u.tile_end - 1; ok && tile >= u.tile; --tile, ++i) {
                const int b = i & 1;
                const uint32_t ph = ((i >> 1) & 1) ^ 1;
                const Tile tl = qt_tile(u, tile);
                const int sg = it % ST;
                const unsigned char *st = stage_p + sg * Sh::kStage;
                const long long slab = (long long)u.b * a.cache.H + u.h;
                if (!tl.nodes)
                    ok = wait(&s.st_full[sg], (it / ST) & 1);
                ok = ok && wait(&s.k_empty[b], ph);
                if (!ok)
                    break;
                if (tl.nodes)
                    qt_nodes<T, D, false>(reinterpret_cast<const T *>(a.staged) + (a.st_k + slab) * a.seq.T * D,
                                          keys_p + b * Sh::kTile, e, tl.valid);
                else
                    qt_expand<D>(st, st + 2 * Sh::kCodes, keys_p + b * Sh::kTile, e, tl.valid);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.k_full[b]);
                if (tile == u.tile_end - 1) {
                    ok = wait(&s.q_empty, (n & 1) ^ 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (e < 4)
                        qt_queries<T, D, false>(a, u, tmem + kQtTmemQ, s.c[n % kQtUnits]);
                    else if (nodes && !std::is_same<T, __half>::value)
                        qt_queries<T, D, true>(a, u, tmem + kQtTmemQ + 64, nullptr);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&s.q_full);
                }
                ok = wait(&s.v_empty[b], ph);
                if (!ok)
                    break;
                if (tl.nodes)
                    odd = qt_nodes<T, D, true>(reinterpret_cast<const T *>(a.staged) + (a.st_v + slab) * a.seq.T * D,
                                               values_p + b * Sh::kTile, e, tl.valid);
                else
                    qt_expand<D>(st + Sh::kCodes, st + 2 * Sh::kCodes + Sh::kScales, values_p + b * Sh::kTile, e, tl.valid);
                if (lane == 0 && tile == u.tile_end - 1)
                    s.odd[n % kQtUnits][e] = odd;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.v_full[b]);
                    if (!tl.nodes)
                        mbar_arrive(&s.st_empty[sg]);
                }
                if (!tl.nodes)
                    ++it;
            }
            ++n;
        }
    } else if (warp > kLoadWarp) {  // completes the warpgroup
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        constexpr float kShift = TcType<__half>::kShift, kLazy = TcType<__half>::kLazy;
        const int r = tid;  // row of the unit = TMEM lane
        const uint32_t lanes = (uint32_t)warp << 21, tm_o = tmem + lanes + kQtTmemO;
        uint32_t i = 0, n = 0, joins = 0;
        bool ok = true;
        while (ok && units.next(u)) {
            const bool real = r < u.n_rows;
            const bool busy = __any_sync(0xFFFFFFFFu, real);
            const int tok = (u.row0 + r) / a.G;
            float m = -INFINITY, l = 0.0f, cq = 0.0f;
            for (int tile = u.tile_end - 1; tile >= u.tile; --tile, ++i) {
                const int b = i & 1;
                ok = wait(&s.s_full[b], (i >> 1) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const bool first = tile == u.tile_end - 1;
                // every phase of pv_done is waited for, at the latest before
                // the tile is handed over: a parity says nothing of older ones
                bool seen = first;
                if (first)
                    cq = *reinterpret_cast<const volatile float *>(&s.c[n % kQtUnits][r]);
                if (busy) {
                    const Tile tl = qt_tile(u, tile);
                    const float c = tl.nodes ? a.scale_log2 : cq;
                    const uint32_t tm_s = tmem + lanes + b * 128;
                    const int nch = (tl.valid + 31) / 32, lim = tl.valid;
                    uint32_t s0[32], s1[32];
                    uint64_t bits = 0;  // nodes that the row sees
                    const bool plain = !tl.nodes && lim == kKeys;
                    float mx;
                    if (plain) {
                        tc_load(tm_s, s0);
                        tc_ld32(tm_s + 32, s1);
                        mx = max32(s0);
                        tc_loaded(s1);
                        tc_ld32(tm_s + 64, s0);
                        mx = fmaxf(mx, max32(s1));
                        tc_loaded(s0);
                        tc_ld32(tm_s + 96, s1);
                        mx = fmaxf(mx, max32(s0));
                        tc_loaded(s1);
                        mx = fmaxf(mx, max32(s1));
                    } else {
                        if (tl.nodes) {
                            if (real)
                                bits = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
                            bits &= tl.valid < 64 ? (1ull << tl.valid) - 1 : ~0ull;
                        }
                        mx = -INFINITY;
#pragma unroll 1
                        for (int k = 0; k < nch; ++k) {
                            const uint32_t w = seen32(tl.nodes, bits, lim, k);
                            if (!__any_sync(0xFFFFFFFFu, real && w != 0))
                                continue;
                            tc_load(tm_s + 32 * k, s0);
                            if (__any_sync(0xFFFFFFFFu, real && w != ~0u))
                                hide32(s0, w);
                            mx = fmaxf(mx, max32(s0));
                        }
                    }
                    mx *= c;
                    const bool units_change = !first && tile == u.n_tiles - 2;  // after the nodes' tile
                    if (first) {
                        m = mx;
                    } else if (units_change || __any_sync(0xFFFFFFFFu, mx > m + kLazy)) {
                        float f = 1.0f;
                        if (mx > m + kLazy) {
                            f = exp2_sfu(m - mx);  // 0 when nothing was seen before
                            m = mx;
                        }
                        l *= f;
                        if (units_change)
                            f *= 1.0f / kQ4Units;
                        ok = wait(&s.pv_done, (i - 1) & 1);
                        seen = true;
                        if (!ok)
                            break;
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[16];
                            tc_ld16(tm_o + k, o);
                            tc_wait_ld();
                            tc_pin<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st16(tm_o + k, o);
                        }
                        if (plain)
                            tc_load(tm_s + 96, s1);  // s0, s1 may have been given up for O
                    }
                    const float m0 = m == -INFINITY ? 0.0f : m;
                    const uint64_t c2 = pair(c, c), m2 = pair(kShift - m0, kShift - m0);
                    uint64_t sum[2] = {0, 0};
                    // weights of chunk k, in the upper half of the scores'
                    // columns: from the top down they replace scores that
                    // have been read for the last time
                    auto weigh32 = [&](const uint32_t *v, int k) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            unpair(fma2(pair(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, m2), x0, x1);
                            const float p0 = exp2_sfu(x0), p1 = exp2_sfu(x1);
                            sum[e & 1] = add2(sum[e & 1], pair(p0, p1));
                            if (!std::is_same<T, __half>::value && tl.nodes)
                                pk[e] = TcType<T>::pack(p0, p1);
                            else
                                pk[e] = TcType<__half>::pack(p0, p1);
                        }
                        tc_st16(tm_s + kQtTmemP + 16 * k, pk);
                    };
                    if (plain) {
                        tc_ld32(tm_s + 64, s0);
                        weigh32(s1, 3);
                        tc_loaded(s0);
                        tc_ld32(tm_s + 32, s1);
                        weigh32(s0, 2);
                        tc_loaded(s1);
                        tc_ld32(tm_s, s0);
                        weigh32(s1, 1);
                        tc_loaded(s0);
                        weigh32(s0, 0);
                    } else {
#pragma unroll 1
                        for (int k = nch - 1; k >= 0; --k) {
                            const uint32_t w = seen32(tl.nodes, bits, lim, k);
                            if (!__any_sync(0xFFFFFFFFu, real && w != 0)) {
                                uint32_t none[16] = {};
                                tc_st16(tm_s + kQtTmemP + 16 * k, none);
                                continue;
                            }
                            tc_load(tm_s + 32 * k, s0);
                            if (__any_sync(0xFFFFFFFFu, real && w != ~0u))
                                hide32(s0, w);
                            weigh32(s0, k);
                        }
                    }
                    {
                        float x0, x1;
                        unpair(add2(sum[0], sum[1]), x0, x1);
                        l += x0 + x1;
                    }
                    tc_wait_st();
                }
                if (!seen) {
                    ok = wait(&s.pv_done, (i - 1) & 1);
                    if (!ok)
                        break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.p_full[b]);
            }
            if (!ok)
                break;
            const bool whole = u.n_parts == 1;
            float *slot = whole ? nullptr : part_slot<kQtRows>(a, blockIdx.x, u.part);
            ok = wait(&s.pv_done, (i - 1) & 1);
            if (!ok)
                break;
            tc_fence_after();
            if (busy) {
                const float to = u.tile < u.n_tiles - 1 ? kQ4Units : 1.0f;  // O's units
                const float f = !whole ? to : l > 0.0f || l != l ? to / l : 0.0f;
                bool any_odd = false;
                if (u.tile_end == u.n_tiles)
#pragma unroll
                    for (int k = 0; k < kQtExpand; ++k)
                        any_odd |= *reinterpret_cast<const volatile int *>(&s.odd[n % kQtUnits][k]) != 0;
                T *dst = real ? reinterpret_cast<T *>(a.out) + row_place(a, u, r) : nullptr;
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    uint32_t o[32];
                    tc_load(tm_o + k, o);
                    in_order32(o);
                    if (any_odd && real) {
                        uint32_t y[32];  // rare; the call keeps only this copy in memory
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            y[e] = o[e];
                        qt_put_back32<T, D>(a, u, tok, k, y);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = y[e];
                    }
                    if (!real)
                        continue;
                    if (whole) {
                        store_row32<T>(dst + k, o, f);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            __stcg(reinterpret_cast<float4 *>(slot + part_quad<kQtRows>((k + e) / 4, r)),
                                   make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f,
                                               __uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f));
                    }
                }
                if (real && !whole) {
                    __stcg(slot + (size_t)kQtRows * D + r, m);
                    __stcg(slot + (size_t)kQtRows * D + kQtRows + r, l);
                }
            }
            tc_fence_before();
            if (!whole) {
                __threadfence();
                mbar_arrive(&s.joined);
                ok = wait(&s.joined, joins++ & 1);
                if (!ok)
                    break;
                if (tid == 0) {
                    int *cnt = part_counter(a, u.first_cta);
                    s.last = atomicAdd(cnt, 1) == u.n_parts - 1;
                    if (s.last)
                        *cnt = 0;
                }
                __syncwarp();
                mbar_arrive(&s.joined);
                ok = wait(&s.joined, joins++ & 1);
                if (!ok)
                    break;
                if (s.last) {
                    __threadfence();
                    ok = join_parts<T, kQtRows>(a, u, tid, 128, [&] {
                        __threadfence();
                        mbar_arrive(&s.joined);
                        return wait(&s.joined, joins++ & 1);
                    });
                    if (!ok)
                        break;
                }
            }
            ++n;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (s.abort) {
        if (warp == kLoadWarp && lane == 0)
            await_copies<ST>(s.st_full, s.asked);
        if (warp == kMmaWarp) {
            await_products(&s.settled);
            give_up(a);
        }
    }
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

namespace {

template <typename T, int D>
cudaError_t launch_qt(const AttendQ4Args &a, cudaStream_t st)
{
    const cudaError_t e = cudaFuncSetAttribute(attend_q4_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               QtShape<D>::kSmem);
    if (e != cudaSuccess)
        return e;
    attend_q4_tc_kernel<T, D><<<kAttendCtas, kQtThreads, QtShape<D>::kSmem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_q4_tc(const AttendQ4Args &a, spec_dtype dt, cudaStream_t st)
{
    if (a.pool.D == 64)
        return dt == SPEC_BF16 ? launch_qt<__nv_bfloat16, 64>(a, st) : launch_qt<__half, 64>(a, st);
    return dt == SPEC_BF16 ? launch_qt<__nv_bfloat16, 128>(a, st) : launch_qt<__half, 128>(a, st);
}

size_t attend_q4_tc_workspace(int D)
{
    return align256(kPartHead + 2 * kAttendCtas * part_floats<kQtRows>(D) * sizeof(float));
}

}  // namespace spec
