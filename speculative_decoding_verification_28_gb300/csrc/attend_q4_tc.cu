// attend_q4_tc.cu -- attention of a round over pages of 4-bit keys and values on
// the fifth-generation tensor cores, for rounds with many query rows a key head
// (chains of shared heads, trees).
//
//   S = Q K^T in TMEM;  P = 2^(c S - m) in TMEM, fp16;  O += P V in TMEM, fp32
//
// as in attend_tc.cu, with up to 128 query rows a unit.  What is different is
// where the operands come from: pages arrive as codes (cp.async.bulk, a ring of
// tiles of 128 keys), and eight warps, four for keys and four for values, expand them to 16-bit tiles in the
// 128-byte-swizzled form that tcgen05 reads, each 16 bytes of codes (a group,
// one scale) by one thread.  Keys are expanded to the storage type; values to fp16,
// where weights keep 11 bits, and 128 times too small (q4_expand.cuh).  The
// eight dimensions of a word of codes come out in the order 0 4 1 5 2 6 3 7: queries
// and nodes follow that order, and O's columns are put back as they are stored.
// Queries are the first operand of S and lie in TMEM, since shared memory is what
// this kernel is short of.
//
// A part of a unit begins with the nodes, if it has them: fp16 weights keep their
// size, so that O is in its own units until the next tile's pass over it divides it by 128.
//
//   softmax warps   two threads a TMEM lane, each with half of its keys, that
//                   exchange their maxima
//   mma warp        issues S = Q K^T one tile ahead of O += P V, across units
//   load warp       walks over the units; codes and scales of a tile's pages
//   expand warps    tiles of the prefix; the nodes' tile and the queries
//
// With up to 64 rows each row lies in two lanes (COPIES = 2), r and r + 64, of
// which one has the keys 0 .. 63 of every tile and the other the rest: four warps
// would else be idle, and the softmax is the longest chain.  The two
// are joined as parts of a unit are, in shared memory.
//
// What it takes: 256 chains of 9 over 256 .. 4000 keys, 32 / 8 heads of 128, 335 us (96 for
// HBM, 41 of products): a tile of 128 keys 2500 clocks, of which the products of 128 lanes take 1000 and
// shared memory's traffic (64 kB written expanded, 64 read by the products) as much. No pipe is full
// (tensor 32%, ALU 46%, issue 55%): each warp's chain of dependent steps is, expansion first.
#include <type_traits>

#include "paged_units.cuh"
#include "q4_expand.cuh"

namespace spec {

constexpr int kQtLanes = 128;
constexpr int kQtSoftmax = 8;  // warps
constexpr int kQtExpand = 4;   // for keys, and as many for values
constexpr int kQtThreads = 32 * (kQtSoftmax + 4 + 2 * kQtExpand);  // whole warpgroups, see below
constexpr int kQtTmemP = 64;  // columns of a score buffer where its weights begin
constexpr uint32_t kQtTmemO = 256, kQtTmemQ = 384;  // queries of two units, 64 columns each

template <int D>
struct QtShape {
    static constexpr int kPanels = D / 64;
    static constexpr int kPanel = kKeys * 128;
    static constexpr int kTile = kPanels * kPanel;  // bytes of an expanded tile
    static constexpr int kCodes = kKeys * q4_codes(D), kScales = kKeys * q4_scales(D);
    static constexpr int kStage = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
};
// COPIES: of a row, see above
template <int D, int COPIES>
struct QtLayout {
    using Sh = QtShape<D>;
    static constexpr int kStages = D == 64 ? 8 : COPIES == 2 ? 4 : 5;  // what fits (256 chains: 2 366 us, 3 340)
    static constexpr int kOut = COPIES == 2 ? 16 : 32;                 // columns of O that a thread puts out at a time
    static constexpr int kJoinStride = kOut + 4;                       // floats of a row of them in the copies' join
    static constexpr int kJoin = COPIES == 2 ? 2 * 2 * 64 * kJoinStride * 4 : 0;  // bytes
    // two expanded tiles of keys, and of values
    static constexpr int kSmem = 4 * Sh::kTile + kStages * Sh::kStage + kJoin + 1024;
};
template <int STAGES>
struct QtShared {
    uint64_t st_full[STAGES], st_empty[STAGES];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done, joined, settled, never;
    uint64_t pair[4], copies[2];  // of the warps of a quadrant; of two quadrants
    uint32_t asked;  // tiles that were copied in all
    uint32_t scan[32];
    Run run;
    PagedRing units;
    uint32_t tmem;
    int abort, last;
    float top[2][2][kQtLanes];       // maxima of both halves of a lane's keys, of two tiles
    float m[kQtLanes], l[2][kQtLanes];
    int odd[kUnitRing][kQtExpand];      // whether a value of the nodes is not finite
};

// whether a phase has ended, at once
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// A part's tiles in the order in which they are taken: the last, the nodes', first.
__device__ __forceinline__ Tile qt_tile(const PagedUnit &u, int tile)
{
    Tile t;
    t.nodes = tile == u.n_tiles - 1;
    t.valid = t.nodes ? u.n : min(kKeys, u.prefix - tile * kKeys);
    t.masked = t.nodes;
    return t;
}

// where 16 bytes `chunk` of a row's 128 in a swizzled panel lie
__device__ __forceinline__ int swizzled(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// A tile's keys or values (KEYS), expanded by one warp of kQtExpand, in a short
// loop: every role's code competes for the instruction cache (unrolled four times
// 369 us for 256 chains and 140 for 32 trees of 64, against 340 and 114).
template <typename T, int D, bool KEYS>
__device__ __forceinline__ void qt_expand(const unsigned char *stage, unsigned char *to, int warp, int valid)
{
    using Sh = QtShape<D>;
    using S = typename std::conditional<KEYS && !std::is_same<T, __half>::value, Scale2Bf16, Scale2>::type;
    // eight lanes take two groups of four keys, of the first panel for two keys and of the
    // second for two (D = 128): neither what they read nor what they write collides
    const int lane = threadIdx.x & 31, half = lane & 1, k2 = lane >> 1 & 3;
    constexpr int kEach = D == 128 ? 8 : 16;  // keys of a step
    const int panel = D == 128 ? (lane >> 3 ^ lane >> 2) & 1 : 0, group = 2 * panel + half;
    const int key0 = warp * (kKeys / kQtExpand) + (D == 128 ? lane >> 4 << 2 : lane >> 3 << 2) + k2;
    const unsigned char *codes = stage + (KEYS ? 0 : Sh::kCodes) + key0 * q4_codes(D) + group * 16;
    const unsigned char *scales = stage + 2 * Sh::kCodes + (KEYS ? 0 : Sh::kScales) + key0 * q4_scales(D) + group;
    unsigned char *dst = to + panel * Sh::kPanel + key0 * 128;
    int at[4];  // steps are multiples of eight keys apart, which leaves the swizzle as it is
#pragma unroll
    for (int k = 0; k < 4; ++k)
        at[k] = ((4 * half + k) ^ (key0 & 7)) << 4;
#pragma unroll 1
    for (int i = 0; i < kKeys / kQtExpand; i += kEach) {
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + i * q4_codes(D));
        uint32_t b = scales[i * q4_scales(D)];
        if (!KEYS && valid < kKeys && key0 + i >= valid)  // products read these rows; keys' scores are hidden
            b = 0;
        const S s(std::is_same<S, Scale2>::value ? b * 0x00800080u : b);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
            q4_expand(x[k], s, y);
            *reinterpret_cast<uint4 *>(dst + at[k] + i * 128) = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
}

// The nodes' keys or values, by one warp; true: some value was not finite (and
// is 0 now, `clean`).
template <typename T, int D>
__device__ __forceinline__ bool qt_nodes(const T *rows, unsigned char *to, int warp, int n, bool clean)
{
    constexpr int kChunks = D / 8;
    const int lane = threadIdx.x & 31, end = (n + 15) & ~15;
    bool odd = false;
#pragma unroll 2
    for (int i = warp * 32 + lane; i < end * kChunks; i += 32 * kQtExpand) {
        const int key = i / kChunks, c = i - key * kChunks;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (key < n)
            x = __ldg(reinterpret_cast<const uint4 *>(rows + (size_t)key * D) + c);
        uint32_t y[4];
        pairs_of(x, y);
        if (clean) {
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

// A unit's queries to TMEM, a thread a lane.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void qt_queries(const AttendArgs &a, const PagedUnit &u, uint32_t tmem)
{
    const int row = (threadIdx.x & 127) & (ROWS - 1);
    const uint32_t lanes = (threadIdx.x >> 5 & 3) << 21;
    const bool real = row < u.n_rows;
    const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.q) + row_place(a, u, real ? row : 0));
#pragma unroll
    for (int h = 0; h < D / 8; h += 8) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = real ? __ldg(p + h + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pairs_of(x[k + i], y + 4 * i);
            tc_st16(tmem + lanes + 4 * (h + k), y);
        }
    }
    tc_wait_st();
    tc_fence_before();
}

// Columns in the order of the expanded words -> as they are.
template <int W>
__device__ __forceinline__ void put_in_order(uint32_t *o)
{
#pragma unroll
    for (int w = 0; w < W; w += 8) {
        const uint32_t x[8] = {o[w], o[w + 2], o[w + 4], o[w + 6], o[w + 1], o[w + 3], o[w + 5], o[w + 7]};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[w + i] = x[i];
    }
}

// W columns of a row's half of O
template <int W>
__device__ __forceinline__ void load_row(uint32_t addr, uint32_t *o)
{
    if constexpr (W == 32) {
        tc_load(addr, o);
    } else {
        tc_ld16(addr, o);
        tc_wait_ld();
        tc_pin<16>(o);
    }
}
// ... times f, rounded, to dst
template <typename T, int W>
__device__ __forceinline__ void store_row(T *dst, const uint32_t *o, float f)
{
    if constexpr (W == 32) {
        store_row32<T>(dst, o, f);
    } else {
#pragma unroll
        for (int e = 0; e < W; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = TcType<T>::pack(__uint_as_float(o[e + 2 * i]) * f, __uint_as_float(o[e + 2 * i + 1]) * f);
            *reinterpret_cast<uint4 *>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Adds what is not finite among the nodes' values to columns col .. col + W - 1
// of a row that sees it; its weights are positive, so that it stays as it is.
template <typename T, int D, int W>
__device__ __noinline__ void qt_put_back(const AttendArgs &a, const PagedUnit &u, int row, int col, uint32_t *o)
{
    const T *values = reinterpret_cast<const T *>(a.staged) + (a.st_v + (long long)u.b * a.cache.H + u.h) * a.seq.T * D;
    const uint64_t bits = row_nodes(a, u, row);
    for (int key = 0; key < u.n; ++key)
        if (bits >> key & 1)
            for (int e = 0; e < W; ++e) {
                const float f = Storage<T>::at(values + (size_t)key * D, col + e);
                if (!(fabsf(f) <= 3.4e38f))
                    o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
            }
}

template <typename T, int D, int COPIES>
__global__ void __launch_bounds__(kQtThreads, 1) attend_q4_tc_kernel(const __grid_constant__ AttendQ4Args x)
{
    using Sh = QtShape<D>;
    using Lay = QtLayout<D, COPIES>;
    constexpr int ST = Lay::kStages;
    extern __shared__ unsigned char dyn[];
    __shared__ QtShared<ST> s;
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    unsigned char *keys_p = base, *values_p = base + 2 * Sh::kTile, *stage_p = base + 4 * Sh::kTile;
    float *join_p = reinterpret_cast<float *>(stage_p + ST * Sh::kStage);
    const AttendArgs &a = x.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kRows = kQtLanes / COPIES;  // of a unit
    // A unit's start and end cost about two tiles.  Counted as none / 1 / 2 / 4, us: 256 chains of 9 374 / 357 / 335 /
    // 339, 32 trees of 64 nodes 130 / 120 / 115 / 114, of heads of 64 105 / 97 / 92 / 94; 64 chains of 20 rows 115 /
    // 104 / 100 / 102, 32 of 80 82 / 76 / 72 / 73, 128 of 36 rows and heads of 64 171 / 161 / 154 / 158.
    const UnitShape<2> sh{kKeys, kRows, a.G};
    constexpr int kMmaWarp = kQtSoftmax, kLoadWarp = kMmaWarp + 1, kFirstExpand = kMmaWarp + 4;
    constexpr bool kHalf = std::is_same<T, __half>::value;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&s.st_full[i], 1);
            mbar_init(&s.st_empty[i], 2 * kQtExpand);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], kQtExpand);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_full[i], kQtExpand);
            mbar_init(&s.v_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.q_full[i], kQtExpand);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.p_full[i], kQtSoftmax);
            mbar_init(&s.copies[i], 4);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(&s.pair[i], 2);
        units_init(s.units, kQtSoftmax + 1 + 2 * kQtExpand);
        mbar_init(&s.pv_done, 1);
        mbar_init(&s.joined, 32 * kQtSoftmax);
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
    auto get = [&](uint32_t n, PagedUnit &u) { return units_get(s.units, n, u, &s.abort, limit); };
    PagedUnit u;

    // 640 threads launch with 96 registers each (61440); the softmax keeps 120, the
    // others 80 (256 * 120 + 384 * 80 = 61440; 256 chains 340 us, with 104 and 88 350, with 136
    // and 64 for the expansion 365)
    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        UnitWalk<UnitShape<2>> walk(a, sh, s.run);
        AttendUnit w{};
        TileCopies<D, kKeys> copies(x);
        uint32_t it = 0, n = 0;
        bool ok = true;
        while (ok && walk.next(w)) {
            ok = units_put(s.units, n++, &w, &s.abort, limit);
            prefetch_unit<T, D>(a, w);
            copies.begin(w);
            for (int tile = min(w.tile_end, w.n_tiles - 1) - 1; ok && tile >= w.tile; --tile, ++it) {
                const int sg = it % ST, page = copies.template page_of<false>(tile);
                ok = wait(&s.st_empty[sg], ((it / ST) & 1) ^ 1);
                if (!ok)
                    break;
                copies.issue(tile, page, stage_p + sg * Sh::kStage, &s.st_full[sg]);
            }
        }
        if (ok)
            units_put(s.units, n, nullptr, &s.abort, limit);
        if (lane == 0)
            s.asked = it;
        paged_flags(x, sh, s.run);
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------------- mma
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const uint32_t one = elect_one();
        const uint32_t keys = smem_addr(keys_p), values = smem_addr(values_p);
        auto commit = [&](uint64_t *bar) {
            if (one)
                tc_commit(bar);
        };
        // scores run one tile ahead of weights, across units
        PagedUnit w;
        uint32_t i = 0, is = 0, n = 0, nq = 0;  // tiles weighed and scored, units weighed and scored
        bool have = get(0, w);
        int wt = w.tile_end - 1;
        bool ok = true;
        // (a try_wait would sleep on one barrier while the other's phase ends: 349 us for 256 chains, against 343)
        auto ready = [&](uint64_t *bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, mbar_test(bar, parity)); };
        auto score_next = [&]() {
            const int b = is & 1;
            const Tile tl = qt_tile(w, wt);
            tc_fence_after();
            const uint32_t ides = tc_idesc<T>(min(kKeys, (tl.valid + 15) & ~15), false);
            const uint32_t q = tmem + kQtTmemQ + (nq & 1) * 64, kd = operand(keys + b * Sh::kTile, 16);
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
                mma_ts(one, tmem + b * 128, q + c * 8, kd + (((c / 4) * Sh::kPanel + (c % 4) * 32) >> 4), ides, c > 0);
            commit(&s.s_full[b]);
            commit(&s.k_empty[b]);
            ++is;
            if (--wt < w.tile) {
                commit(&s.q_empty[nq & 1]);
                ++nq;
                have = get(nq, w);
                wt = w.tile_end - 1;
            }
        };
        auto can_score = [&]() -> bool {
            return (wt < w.tile_end - 1 || ready(&s.q_full[nq & 1], (nq >> 1) & 1)) && ready(&s.k_full[is & 1], (is >> 1) & 1);
        };
        if (have) {
            ok = wait(&s.q_full[0], 0) && wait(&s.k_full[0], 0);
            if (ok)
                score_next();
        }
        for (; ok && get(n, u); ++n) {
            for (int tile = u.tile_end - 1; ok && tile >= u.tile; --tile, ++i) {
                const int b = i & 1;
                const Tile tl = qt_tile(u, tile);
                // the next tile's scores and this one's product, whichever can go first:
                // a unit's last product does not wait for the next unit's keys
                bool score = have, weigh = true;
                const long long t0 = clock64();
                while (ok && (score || weigh)) {
                    if (score && can_score()) {
                        score_next();
                        score = false;
                    } else if (weigh && ready(&s.p_full[b], (i >> 1) & 1) && ready(&s.v_full[b], (i >> 1) & 1)) {
                        tc_fence_after();
                        const uint32_t ides = tl.nodes ? tc_idesc<T>(D, true) : tc_idesc<__half>(D, true);
                        const uint32_t vd = operand(values + b * Sh::kTile, Sh::kPanel), p = tmem + b * 128 + kQtTmemP;
                        mma_ts(one, tmem + kQtTmemO, p, vd, ides, tile < u.tile_end - 1);
                        for (int c = 1; c < (tl.valid + 15) / 16; ++c)
                            mma_ts(one, tmem + kQtTmemO, p + c * 8, vd + c * (2048 >> 4), ides, 1);
                        commit(&s.v_empty[b]);
                        commit(&s.pv_done);
                        weigh = false;
                    } else if (clock64() - t0 > limit || *reinterpret_cast<volatile int *>(&s.abort)) {
                        *reinterpret_cast<volatile int *>(&s.abort) = 1;
                        ok = false;
                    }
                    ok = __all_sync(0xFFFFFFFFu, ok);
                }
            }
            units_done(s.units, n);
        }
    } else if (warp >= kFirstExpand) {
        // ----------------------------------------------------------- expand
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // Keys and values each at their own pace: a tile's keys are wanted as soon as
        // the scores before are formed, its values two products later.
        const int e = warp & 3;
        const bool keys = warp < kFirstExpand + kQtExpand;
        uint64_t *full = keys ? s.k_full : s.v_full, *empty = keys ? s.k_empty : s.v_empty;
        unsigned char *tiles = keys ? keys_p : values_p;
        uint32_t i = 0, it = 0, n = 0;  // tiles, tiles of the prefix, units
        bool ok = !a.starve || wait(&s.never, 0);
        for (; ok && get(n, u); ++n) {
            for (int tile = u.tile_end - 1; ok && tile >= u.tile; --tile, ++i) {
                const int b = i & 1;
                const Tile tl = qt_tile(u, tile);
                const int sg = it % ST;
                unsigned char *to = tiles + b * Sh::kTile;
                if (!tl.nodes)
                    ok = wait(&s.st_full[sg], (it / ST) & 1);
                ok = ok && wait(&empty[b], ((i >> 1) & 1) ^ 1);
                if (!ok)
                    break;
                bool odd = false;
                if (tl.nodes) {
                    const long long slab = (keys ? a.st_k : a.st_v) + (long long)u.b * a.cache.H + u.h;
                    odd = qt_nodes<T, D>(reinterpret_cast<const T *>(a.staged) + slab * a.seq.T * D, to, e, tl.valid, !keys);
                } else if (keys) {
                    qt_expand<T, D, true>(stage_p + sg * Sh::kStage, to, e, tl.valid);
                } else {
                    qt_expand<T, D, false>(stage_p + sg * Sh::kStage, to, e, tl.valid);
                }
                if (!keys && lane == 0 && tile == u.tile_end - 1)
                    s.odd[n % kUnitRing][e] = odd;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&full[b]);
                    if (!tl.nodes)
                        mbar_arrive(&s.st_empty[sg]);
                }
                if (!tl.nodes)
                    ++it;
                if (keys && tile == u.tile_end - 1) {
                    ok = wait(&s.q_empty[n & 1], ((n >> 1) & 1) ^ 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    qt_queries<T, D, kRows>(a, u, tmem + kQtTmemQ + (n & 1) * 64);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&s.q_full[n & 1]);
                }
            }
            units_done(s.units, n);
        }
    } else if (warp > kLoadWarp) {  // completes the warpgroup
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        constexpr float kLazy = TcType<__half>::kLazy;
        constexpr int kCols = 64 / COPIES;  // a thread's keys of a tile
        const int side = warp >> 2, quad = warp & 3;
        const int at = tid & 127, r = at & (kRows - 1), copy = COPIES == 2 ? at >> 6 : 0;  // TMEM lane, row, copy
        const int col = COPIES == 2 ? 64 * copy + 32 * side : 64 * side;                   // first key
        const uint32_t lanes = (uint32_t)quad << 21, tm_o = tmem + lanes + kQtTmemO + side * (D / 2);
        uint32_t i = 0, n = 0, joins = 0, pairs = 0, meets = 0;
        bool ok = true;
        // both warps of a quadrant, and those of the quadrants of both copies
        auto meet = [&](uint64_t *bar, uint32_t &count) -> bool {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
            return wait(bar, count++ & 1);
        };
        for (; ok && get(n, u); ++n) {
            const bool real = r < u.n_rows;
            const bool busy = __any_sync(0xFFFFFFFFu, real);
            float m = -INFINITY, l = 0.0f;
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
                if (busy) {
                    const Tile tl = qt_tile(u, tile);
                    const float c = kHalf && !tl.nodes ? a.scale_log2 * kQ4Units : a.scale_log2;
                    const uint32_t tm_s = tmem + lanes + b * 128, tm_p = tm_s + kQtTmemP + col / 2;
                    uint32_t x[kCols / 32][32];
                    float mx = -INFINITY;
                    uint64_t bits = 0;  // nodes that the row sees
                    if (tl.nodes && real)
                        bits = row_nodes(a, u, r);
#pragma unroll
                    for (int k = 0; k < kCols / 32; ++k)
                        tc_ld32(tm_s + col + 32 * k, x[k]);
#pragma unroll
                    for (int k = 0; k < kCols / 32; ++k) {
                        if (k == 0)
                            tc_wait_ld();
                        tc_pin<32>(x[k]);
                        if (tl.valid < kKeys)  // at most 64 nodes, so all in the first two words
                            hide32(x[k], tl.nodes && col >= 64 ? 0u : seen32(tl.nodes, bits, tl.valid, col / 32 + k));
                        mx = fmaxf(mx, max32(x[k]));
                    }
                    // the lane's maximum; both threads have read their scores by then,
                    // so that weights may take the upper half of their columns
                    s.top[b][side][at] = mx;
                    ok = meet(&s.pair[quad], pairs);
                    if (!ok)
                        break;
                    mx = fmaxf(mx, *reinterpret_cast<const volatile float *>(&s.top[b][side ^ 1][at])) * c;
                    // fp16 weights of the nodes stay as large as the others', so that their
                    // O is in its own units; bf16 ones can be 128 times smaller
                    const bool units_change = kHalf && !first && tile == u.n_tiles - 2;
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
                        for (int k = 0; k < D / 2; k += 16) {
                            uint32_t o[16];
                            tc_ld16(tm_o + k, o);
                            tc_wait_ld();
                            tc_pin<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st16(tm_o + k, o);
                        }
                    }
                    const bool small = !kHalf && tl.nodes;
                    const float shift = (small ? 4.0f : TcType<__half>::kShift) - (m == -INFINITY ? 0.0f : m);
                    const uint64_t c2 = pair(c, c), m2 = pair(shift, shift);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int k = 0; k < kCols / 32; ++k) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            unpair(fma2(pair(__uint_as_float(x[k][2 * e]), __uint_as_float(x[k][2 * e + 1])), c2, m2), x0, x1);
                            const float p0 = exp2_sfu(x0), p1 = exp2_sfu(x1);
                            sum[e & 1] = add2(sum[e & 1], pair(p0, p1));
                            pk[e] = small ? TcType<T>::pack(p0, p1) : TcType<__half>::pack(p0, p1);
                        }
                        tc_st16(tm_p + 16 * k, pk);
                    }
                    if (COPIES == 2) {  // the other copy's keys
                        uint32_t none[16] = {};
                        tc_st16(tm_s + kQtTmemP + (col ^ 64) / 2, none);
                    }
                    {
                        float x0, x1;
                        unpair(add2(sum[0], sum[1]), x0, x1);
                        l = fmaf(x0 + x1, small ? kQ4Units : 1.0f, l);
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
            float *slot = whole ? nullptr : part_slot<kRows>(a, blockIdx.x, u.part);
            ok = wait(&s.pv_done, (i - 1) & 1);
            if (!ok)
                break;
            tc_fence_after();
            if (busy) {
                const float units = kHalf && u.tile == u.n_tiles - 1 ? 1.0f : kQ4Units;  // O's
                // the row's sum, over both sides and copies, under a common maximum
                s.l[side][at] = l;
                if (side == 0)
                    s.m[at] = m;
                ok = COPIES == 2 ? meet(&s.copies[quad & 1], meets) : meet(&s.pair[quad], pairs);
                if (!ok)
                    break;
                const volatile float *vl = &s.l[0][0], *vm = s.m;
                float f = units;
                l = vl[at] + vl[kQtLanes + at];
                if (COPIES == 2) {
                    const float m1 = vm[at ^ 64], l1 = vl[at ^ 64] + vl[kQtLanes + (at ^ 64)];
                    const float top = fmaxf(m, m1), m0 = top == -INFINITY ? 0.0f : top;
                    const float f0 = exp2f(m - m0);
                    l = fmaf(f0, l, exp2f(m1 - m0) * l1);
                    m = top;
                    f *= f0;
                }
                bool any_odd = false;
                if (u.tile_end == u.n_tiles)
#pragma unroll
                    for (int k = 0; k < kQtExpand; ++k)
                        any_odd |= *reinterpret_cast<const volatile int *>(&s.odd[n % kUnitRing][k]) != 0;
                const float inv = !whole ? 1.0f : l > 0.0f || l != l ? 1.0f / l : 0.0f;
                // Each copy puts out half of this side's columns and gives the other half
                // away, a few at a time: the ring needs the room.
                constexpr int kMine = D / 2 / COPIES, W = Lay::kOut;
                const int out0 = copy * kMine, d0 = side * (D / 2) + out0;
                float *give = join_p + ((side * 2 + (copy ^ 1)) * 64 + r) * Lay::kJoinStride;
                const float *take = join_p + ((side * 2 + copy) * 64 + r) * Lay::kJoinStride;
                T *dst = real ? reinterpret_cast<T *>(a.out) + row_place(a, u, r) + d0 : nullptr;
#pragma unroll 1
                for (int k = 0; k < kMine; k += W) {
                    uint32_t o[W];
                    if (COPIES == 2) {
                        load_row<W>(tm_o + (out0 ^ kMine) + k, o);
                        if (k > 0)  // what was given before has been read
                            ok = meet(&s.copies[quad & 1], meets);
#pragma unroll
                        for (int e = 0; e < W; e += 4)
                            *reinterpret_cast<float4 *>(give + e) =
                                make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f,
                                            __uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
                        ok = ok && meet(&s.copies[quad & 1], meets);
                        if (!ok)
                            break;
                    }
                    load_row<W>(tm_o + out0 + k, o);
#pragma unroll
                    for (int e = 0; e < W; e += 4) {
                        float4 y = make_float4(0, 0, 0, 0);
                        if (COPIES == 2)
                            y = *reinterpret_cast<const float4 *>(take + e);
                        o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), f, y.x));
                        o[e + 1] = __float_as_uint(fmaf(__uint_as_float(o[e + 1]), f, y.y));
                        o[e + 2] = __float_as_uint(fmaf(__uint_as_float(o[e + 2]), f, y.z));
                        o[e + 3] = __float_as_uint(fmaf(__uint_as_float(o[e + 3]), f, y.w));
                    }
                    put_in_order<W>(o);
                    if (any_odd && real) {
                        uint32_t y[W];  // rare; the call keeps only these copies in memory
                        const PagedUnit v = u;
#pragma unroll
                        for (int e = 0; e < W; ++e)
                            y[e] = o[e];
                        qt_put_back<T, D, W>(a, v, r, d0 + k, y);
#pragma unroll
                        for (int e = 0; e < W; ++e)
                            o[e] = y[e];
                    }
                    if (real && whole) {
                        store_row<T, W>(dst + k, o, inv);
                    } else if (real) {
#pragma unroll
                        for (int e = 0; e < W; e += 4)
                            __stcg(reinterpret_cast<uint4 *>(slot + part_quad<kRows>((d0 + k + e) / 4, r)),
                                   make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
                if (real && !whole && side == 0 && copy == 0) {
                    __stcg(slot + (size_t)kRows * D + r, m);
                    __stcg(slot + (size_t)kRows * D + kRows + r, l);
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
                    ok = join_parts<T, kRows>(a, join_unit(a, u), tid, 32 * kQtSoftmax, [&] {
                        __threadfence();
                        mbar_arrive(&s.joined);
                        return wait(&s.joined, joins++ & 1);
                    });
                    if (!ok)
                        break;
                }
            }
            units_done(s.units, n);
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

template <typename T, int D, int COPIES>
cudaError_t launch_qt(const AttendQ4Args &a, cudaStream_t st)
{
    constexpr int smem = QtLayout<D, COPIES>::kSmem;
    const cudaError_t e =
        cudaFuncSetAttribute(attend_q4_tc_kernel<T, D, COPIES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    attend_q4_tc_kernel<T, D, COPIES><<<kAttendCtas, kQtThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_qt_t(const AttendQ4Args &a, cudaStream_t st)
{
    // (64 chains of 20 rows 101 us, with one copy 119; 256 of 36 340, 403)
    const bool few = a.a.seq.T * a.a.G <= kQtLanes / 2;
    if (a.pool.D == 64)
        return few ? launch_qt<T, 64, 2>(a, st) : launch_qt<T, 64, 1>(a, st);
    return few ? launch_qt<T, 128, 2>(a, st) : launch_qt<T, 128, 1>(a, st);
}

}  // namespace

cudaError_t launch_attend_q4_tc(const AttendQ4Args &a, spec_dtype dt, cudaStream_t st)
{
    return dt == SPEC_BF16 ? launch_qt_t<__nv_bfloat16>(a, st) : launch_qt_t<__half>(a, st);
}

size_t attend_q4_tc_workspace(int D)
{
    return align256(kPartHead + 2 * kAttendCtas * part_floats<kQtLanes>(D) * sizeof(float));
}

}  // namespace spec
