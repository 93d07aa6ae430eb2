// attend_tc.cu -- attention on the tensor cores (tcgen05), for bf16 and fp16
// caches with heads of 64 or 128.
//
//   S = Q K^T in TMEM;  P = 2^(c S - m) in TMEM, rounded to the storage type;
//   O += P V in TMEM, fp32
//
// with one pass over the keys.  A row's m is a running maximum that is only
// moved when a tile's maximum is more than 2^kLazy above it: O and the sum are
// then rescaled.  Between moves the weights exceed 2^kShift by at most 2^kLazy
// (TcType), which costs neither fp32 sums nor 16-bit weights range or precision.
// The weights are rounded to the storage type, by up to half a step (bf16 2^-8,
// fp16 2^-11 of their value), because one tcgen05 product takes both operands in
// one 16-bit type: against 64 bits the results are 1.2 to 1.4 times as far off as
// with fp32 weights, where the result's own rounding remains.  Sums add the fp32
// weights.
//
// A CTA holds NT tiles of 128 query rows of one key head (the G query heads
// that share it, token-major) and streams its keys once:
//   softmax warps   128 NT threads, one per query row: S from TMEM, mask,
//                   maximum, weights and their sum, P to TMEM; at the end O
//   mma warp        issues S = Q K^T and O += P V
//   load warp       TMA of Q, K and V (128-byte swizzle) through a ring
//   guard warp      the last rows of V tiles: places nobody sees are zeroed,
//                   and values that are not finite are taken out where some
//                   rows do not see them (0 * inf would reach those rows)
// NT = 1 (up to 128 query rows): S has two buffers, so the next tile's scores
// form while this tile's weights do.  NT = 2: the two tiles take turns on the
// tensor pipe, one's product runs under the other's softmax.
//
// Bound by the softmax's chain (scores from TMEM, maximum, exponentials,
// weights to TMEM) against the tensor pipe, which is busy 60% of the time: two
// prompts of 8192 tokens, 32 / 8 heads of 128, take 760 us (1.45 PFLOP/s, 0.76
// of a large matrix product).  Slower were: all 128 scores held in registers
// (776 us at the time, against 760), weights handed over by halves (829, 813),
// products of transposed operands and two chains to a CTA for few rows (159 and
// 145 us for chains, against 127).  A round of 32 times 64 nodes, 28 / 4 heads,
// over 500 to 4000 keys takes 109 us: units of some 20 tiles, whose start, end
// and join do not overlap.
#include "tcgen.cuh"

namespace spec {

// ---------------------------------------------------------------------------
// shapes
// ---------------------------------------------------------------------------
constexpr int kShortPrompt = 512;
constexpr int kTmemP = 64;  // columns of a score buffer where its weights begin

template <int D, int NT>
struct TcShape {
    static constexpr int kPanels = D / 64;
    static constexpr int kPanel = kKeys * 128;         // bytes
    static constexpr int kTile = kPanels * kPanel;     // bytes of a Q, K or V tile
    static constexpr int kQBuf = NT == 1 ? 2 : 1;
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kSmem = (kQBuf * NT + kStages) * kTile + 1024;
    static constexpr int kSoftmax = 128 * NT;
    static constexpr int kThreads = kSoftmax + (NT == 2 ? 128 : 96);  // NT = 2: whole warpgroups, see below
    static constexpr int kRows = 128 * NT;
    static constexpr uint32_t kTmemO = 256;
};

template <int STAGES>
struct TcShared {
    uint64_t kv_full[STAGES], kv_empty[STAGES], q_full[2], q_empty[2];
    uint64_t v_ok[STAGES];  // guarded tiles: a stage's next one waits for its own consumption
    uint64_t s_full[2], p_full[2], pv_done[2], joined, settled;
    uint32_t asked_kv, asked_q;  // copies that the load warp asked for in all
    uint32_t scan[16];
    Run run;
    uint32_t tmem;
    int abort, last;
    uint32_t odd[kGuardRing][13];  // keys of the guarded tiles with a value that is not finite; [12]: any
};

// end of the tiles that query tile `t` of the unit needs
template <bool PROMPT, int NT>
__device__ __forceinline__ int tiles_end(const AttendUnit &u, int G, int tile_rows, int t)
{
    if (NT == 1)
        return u.tile_end;
    if (t * tile_rows >= u.n_rows)
        return u.tile;
    if (!PROMPT)
        return u.tile_end;
    const int last = min(u.n_rows, (t + 1) * tile_rows) - 1;
    return (u.seq.prefix + (u.row0 + last) / G + kKeys) / kKeys;
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <typename T, int D, int NT, bool PROMPT>
__global__ void __launch_bounds__(TcShape<D, NT>::kThreads, 1)
    attend_tc_kernel(const AttendArgs a, const __grid_constant__ TcMaps maps, const TcBoxes box)
{
    using Sh = TcShape<D, NT>;
    constexpr int ST = Sh::kStages;
    extern __shared__ unsigned char dyn[];
    __shared__ TcShared<ST> s;
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    unsigned char *ring_p = base + Sh::kQBuf * NT * Sh::kTile;
    const uint32_t q_smem = smem_addr(base), ring = smem_addr(ring_p);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile_rows = box.tok_tile * a.G;  // query rows of a tile
    const Shape sh{kKeys, NT * tile_rows, a.G};

    AttendUnit first{};
    if (PROMPT && !prompt_unit(a, sh, first))
        return;  // the whole CTA
    constexpr int kMmaWarp = 4 * NT, kLoadWarp = kMmaWarp + 1;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&s.kv_full[i], 1);
            mbar_init(&s.kv_empty[i], 2);  // mma and guard
            mbar_init(&s.v_ok[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.pv_done[i], 1);
        }
        mbar_init(&s.joined, Sh::kSoftmax);
        mbar_init(&s.settled, 1);
        fence_mbar_init();
        s.abort = 0;
        s.run.begin = s.run.end = 0;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (warp == kLoadWarp && lane < 3) {
        const CUtensorMap *m = lane == 0 ? &maps.q : lane == 1 ? &maps.kv : &maps.node;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    if (!PROMPT) {
        __syncthreads();  // run.begin / end above come before find_run's
        find_run<Sh::kThreads>(a, sh, s.scan, &s.run);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;

    // a bounded wait; after one that gave up every role leaves its loop.
    // wait1 is one lane's, wait the whole warp's (its answer is the warp's)
    const long long limit = a.wait_clocks;  // by itself: the waits' reference to all of `a` would put it on the stack
    auto wait1 = [&](uint64_t *bar, uint32_t parity) -> bool { return wait_phase(bar, parity, &s.abort, limit); };
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, wait1(bar, parity));
    };
    Units<PROMPT> units(a, sh, s.run, first, true);
    AttendUnit u{};

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        // A round's walk over units costs the softmax warps registers: 384
        // threads launch with 168 each (64512), those keep 200 and the others
        // 104 (256 * 200 + 128 * 104 = 64512); 149 -> 135 us for trees of 64
        // nodes and 7 heads (208 and 80: 5% slower than this).  A prompt's one unit fits 168.
        if constexpr (NT == 2 && !PROMPT)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (lane == 0) {
            uint32_t it = 0, n = 0;  // tiles of keys and values, of queries
            bool ok = true;
            while (ok && units.next(u)) {
                const int qb = n % Sh::kQBuf;
                ok = wait1(&s.q_empty[qb], ((n / Sh::kQBuf) & 1) ^ 1);
                if (!ok)
                    break;
                mbar_arrive_expect_tx(&s.q_full[qb], NT * Sh::kPanels * box.q_tok * a.G * 128);
                const int tok = (int)u.seq.tok0 + u.row0 / a.G;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int p = 0; p < Sh::kPanels; ++p)
                        tma_load_4d(q_smem + (qb * NT + t) * Sh::kTile + p * Sh::kPanel, &maps.q, p * 64, 0, u.h,
                                    tok + t * box.tok_tile, &s.q_full[qb]);
                ++n;
                for (int tile = u.tile; ok && tile < u.tile_end; ++tile) {
                    const KvBox k = kv_box<Sh::kPanels>(a, maps, box, u, tile, !PROMPT && tile == u.n_tiles - 1);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int sg = it % ST;
                        ok = ok && wait1(&s.kv_empty[sg], ((it / ST) & 1) ^ 1);
                        if (!ok)
                            break;
                        mbar_arrive_expect_tx(&s.kv_full[sg], k.bytes);
#pragma unroll
                        for (int p = 0; p < Sh::kPanels; ++p)
                            tma_load_3d(ring + sg * Sh::kTile + p * Sh::kPanel, k.m, p * 64, k.y, k.z + kv * k.zv,
                                        &s.kv_full[sg]);
                        ++it;
                    }
                }
            }
            s.asked_kv = it;
            s.asked_q = n;
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------------- mma
        if constexpr (NT == 2 && !PROMPT)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        const uint32_t ideo = tc_idesc<T>(D, true);
        uint32_t ok_ph = 0;  // per stage: parity of its guarded uses
        auto wait_guard = [&](int sg) -> bool {
            ok_ph ^= 1u << sg;
            return wait(&s.v_ok[sg], (ok_ph >> sg & 1) ^ 1);
        };
        const uint32_t one = elect_one();
        auto score = [&](uint32_t q, uint32_t k, uint32_t d, int valid) {
            const uint32_t ides = tc_idesc<T>(min(kKeys, (valid + 15) & ~15), false);
            const uint32_t qd = operand(q, 16), kd = operand(k, 16);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const uint32_t o = ((c / 4) * Sh::kPanel + (c % 4) * 32) >> 4;
                mma_ss(one, d, qd + o, kd + o, ides, c > 0);
            }
        };
        auto weigh = [&](uint32_t p, uint32_t v, uint32_t d, int valid, bool add) {
            const uint32_t vd = operand(v, Sh::kPanel);
            mma_ts(one, d, p + kTmemP, vd, ideo, add);
            if (valid > kKeys - 16) {
#pragma unroll
                for (int c = 1; c < kKeys / 16; ++c)
                    mma_ts(one, d, p + kTmemP + c * 8, vd + c * (2048 >> 4), ideo, 1);
            } else {
                for (int c = 1; c < (valid + 15) / 16; ++c)
                    mma_ts(one, d, p + kTmemP + c * 8, vd + c * (2048 >> 4), ideo, 1);
            }
        };
        auto commit = [&](uint64_t *bar) {
            if (one)
                tc_commit(bar);
        };
        if constexpr (NT == 1) {
            // scores run one tile ahead of weights, across units
            Units<PROMPT> ahead(a, sh, s.run, first, true);
            AttendUnit w{};
            bool have = ahead.next(w);
            int wt = w.tile;
            uint32_t i = 0, is = 0, nq = 0;  // tiles weighed, tiles scored, units scored
            bool ok = true;
            auto score_next = [&]() {
                const int qb = nq & 1, sg = (2 * is) % ST;
                if (wt == w.tile)
                    ok = ok && wait(&s.q_full[qb], (nq >> 1) & 1);
                ok = ok && wait(&s.kv_full[sg], ((2 * is) / ST) & 1);
                if (!ok)
                    return;
                tc_fence_after();
                score(q_smem + qb * Sh::kTile, ring + sg * Sh::kTile, tmem + (is & 1) * 128,
                      tile_of<PROMPT>(w, wt).valid);
                commit(&s.s_full[is & 1]);
                commit(&s.kv_empty[sg]);
                ++is;
                if (++wt == w.tile_end) {
                    commit(&s.q_empty[qb]);
                    ++nq;
                    have = ahead.next(w);
                    wt = w.tile;
                }
            };
            if (have)
                score_next();
            while (ok && units.next(u)) {
                for (int tile = u.tile; ok && tile < u.tile_end; ++tile) {
                    if (have)
                        score_next();
                    const int sg = (2 * i + 1) % ST;
                    const Tile tl = tile_of<PROMPT>(u, tile);
                    ok = ok && wait(&s.p_full[i & 1], (i >> 1) & 1) && wait(&s.kv_full[sg], ((2 * i + 1) / ST) & 1);
                    if (ok && guarded(tl))
                        ok = wait_guard(sg);
                    if (!ok)
                        break;
                    tc_fence_after();
                    weigh(tmem + (i & 1) * 128, ring + sg * Sh::kTile, tmem + Sh::kTmemO, tl.valid, tile > u.tile);
                    commit(&s.kv_empty[sg]);
                    commit(&s.pv_done[0]);
                    ++i;
                }
            }
        } else {
            uint32_t i = 0, nq = 0;        // K / V pairs consumed, units
            uint32_t np[NT] = {};          // weight tiles waited for
            bool ok = true;
            while (ok && units.next(u)) {
                int te[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    te[t] = tiles_end<PROMPT, NT>(u, a.G, tile_rows, t);
                const int end = u.tile_end;
                ok = wait(&s.q_full[0], nq & 1) && wait(&s.kv_full[(2 * i) % ST], ((2 * i) / ST) & 1);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (u.tile < te[t]) {
                        score(q_smem + t * Sh::kTile, ring + ((2 * i) % ST) * Sh::kTile, tmem + t * 128,
                              tile_of<PROMPT>(u, u.tile).valid);
                        commit(&s.s_full[t]);
                    }
                commit(&s.kv_empty[(2 * i) % ST]);
                for (int tile = u.tile; ok && tile < end; ++tile, ++i) {
                    const int sv = (2 * i + 1) % ST, sk = (2 * i + 2) % ST;
                    const Tile tl = tile_of<PROMPT>(u, tile);
                    ok = wait(&s.kv_full[sv], ((2 * i + 1) / ST) & 1);
                    if (ok && guarded(tl))
                        ok = wait_guard(sv);
                    if (ok && tile + 1 < end)
                        ok = wait(&s.kv_full[sk], ((2 * i + 2) / ST) & 1);
                    if (!ok)
                        break;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (tile < te[t]) {
                            ok = ok && wait(&s.p_full[t], np[t]++ & 1);
                            if (!ok)
                                break;
                            tc_fence_after();
                            weigh(tmem + t * 128, ring + sv * Sh::kTile, tmem + Sh::kTmemO + t * D, tl.valid,
                                  tile > u.tile);
                            if (tile + 1 == te[t])
                                commit(&s.pv_done[t]);
                        }
                        if (tile + 1 < te[t]) {
                            score(q_smem + t * Sh::kTile, ring + sk * Sh::kTile, tmem + t * 128,
                                  tile_of<PROMPT>(u, tile + 1).valid);
                            commit(&s.s_full[t]);
                        }
                    }
                    commit(&s.kv_empty[sv]);
                    if (tile + 1 < end)
                        commit(&s.kv_empty[sk]);
                }
                commit(&s.q_empty[0]);
                ++nq;
            }
        }
    } else if (warp == kLoadWarp + 2) {  // completes the warpgroup
        if constexpr (NT == 2 && !PROMPT)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    } else if (warp == kLoadWarp + 1) {
        // ------------------------------------------------------------ guard
        if constexpr (NT == 2 && !PROMPT)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        uint32_t i = 0, n = 0;
        bool ok = true;
        while (ok && units.next(u)) {
            uint32_t *odd = s.odd[n % kGuardRing];
            if (lane < 13)
                odd[lane] = 0;
            __syncwarp();
            int g = 0;  // masked tiles of the unit so far
            for (int tile = u.tile; ok && tile < u.tile_end; ++tile, ++i) {
                const Tile tl = tile_of<PROMPT>(u, tile);
                // The guard sees every load of the ring and releases it too, so
                // that no barrier is ever two phases ahead of it
                const int sk = (2 * i) % ST, sg = (2 * i + 1) % ST;
                ok = wait(&s.kv_full[sk], ((2 * i) / ST) & 1);
                if (ok && lane == 0)
                    mbar_arrive(&s.kv_empty[sk]);
                ok = ok && wait(&s.kv_full[sg], ((2 * i + 1) / ST) & 1);
                if (!ok)
                    break;
                if (!guarded(tl)) {
                    if (lane == 0)
                        mbar_arrive(&s.kv_empty[sg]);
                    continue;
                }
                guard_tile<T, Sh::kPanels>(ring_p + sg * Sh::kTile, tl, odd, g);
                if (lane == 0) {
                    mbar_arrive(&s.v_ok[sg]);
                    mbar_arrive(&s.kv_empty[sg]);
                }
            }
            ++n;
        }
    } else {
        // ---------------------------------------------------------- softmax
        if constexpr (NT == 2 && !PROMPT)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        if (!PROMPT && blockIdx.x == 0 && warp == 0)
            flag_if_gave_up(a);
        const int t = NT == 1 ? 0 : warp >> 2;
        const int r = (warp & 3) * 32 + lane;        // row of the tile = TMEM lane
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t tm_o = tmem + lanes + Sh::kTmemO + t * D;
        const float c = a.scale_log2;
        uint32_t i = 0, n = 0, n_done = 0, n_join = 0;  // tiles, units, units with tiles here, joins
        bool ok = true;
        while (ok && units.next(u)) {
            const int ur = t * tile_rows + r;        // row of the unit
            const bool real = r < tile_rows && ur < u.n_rows;
            const bool busy = __any_sync(0xFFFFFFFFu, real);
            const int tok = (u.row0 + ur) / a.G;
            const int end = tiles_end<PROMPT, NT>(u, a.G, tile_rows, t);
            float m = -INFINITY, l = 0.0f;
            for (int tile = u.tile; tile < end; ++tile, ++i) {
                const int x = NT == 1 ? i & 1 : t;
                const uint32_t ph = NT == 1 ? (i >> 1) & 1 : i & 1;
                ok = wait(&s.s_full[x], ph);
                if (!ok)
                    break;
                tc_fence_after();
                // every phase of pv_done is waited for, at the latest before
                // the tile is handed over: a parity says nothing of older ones
                bool seen = NT != 1 || tile == u.tile;
                if (busy) {
                    const Tile tl = tile_of<PROMPT>(u, tile);
                    const uint32_t tm_s = tmem + lanes + x * 128;
                    // The weights take the upper half of the scores' columns.
                    // Chunks of 32 columns are weighed from the top down, each
                    // after the scores that its weights replace, which are
                    // read a second time where registers did not keep them.
                    const int lim = PROMPT ? min(tl.valid, u.seq.prefix + tok + 1 - tile * kKeys) : tl.valid;
                    const bool plain = !tl.nodes && !__any_sync(0xFFFFFFFFu, lim < kKeys);
                    uint32_t s0[32], s1[32], s2[32];
                    float mx;
                    uint64_t bits = 0;  // nodes that the row sees
                    const int nch = (tl.valid + 31) / 32;
                    if (plain) {
                        tc_load(tm_s, s0);
                        tc_ld32(tm_s + 32, s1);
                        mx = max32(s0);
                        tc_loaded(s1);
                        tc_ld32(tm_s + 64, s2);
                        mx = fmaxf(mx, max32(s1));
                        tc_loaded(s2);
                        tc_ld32(tm_s + 96, s1);
                        mx = fmaxf(mx, max32(s2));
                        tc_loaded(s1);
                        mx = fmaxf(mx, max32(s1));
                    } else {
                        if (tl.nodes) {
                            if (real)
                                bits = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
                            bits &= tl.valid < 64 ? (1ull << tl.valid) - 1 : ~0ull;
                        }
                        mx = -INFINITY;
                        // a vote spares chunks that every row of the warp
                        // sees whole, or not at all
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
                    float f = 1.0f;
                    if (tile == u.tile) {
                        m = mx;
                    } else if (__any_sync(0xFFFFFFFFu, mx > m + TcType<T>::kLazy)) {
                        if (mx > m + TcType<T>::kLazy) {
                            f = exp2_sfu(m - mx);  // 0 when nothing was seen before
                            m = mx;
                        }
                        l *= f;
                        if (NT == 1 && !seen) {  // NT = 2: S was scored after the last O += P V
                            ok = wait(&s.pv_done[0], (i - 1) & 1);
                            seen = true;
                        }
                        if (!ok)
                            break;
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < D / 32; ++k) {
                            tc_load(tm_o + 32 * k, s0);
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float x0, x1;
                                unpair(mul2(pair(__uint_as_float(s0[e]), __uint_as_float(s0[e + 1])), pair(f, f)), x0, x1);
                                s0[e] = __float_as_uint(x0);
                                s0[e + 1] = __float_as_uint(x1);
                            }
                            tc_st32(tm_o + 32 * k, s0);
                        }
                    }
                    const float m0 = m == -INFINITY ? 0.0f : m;
                    const uint64_t c2 = pair(c, c), m2 = pair(TcType<T>::kShift - m0, TcType<T>::kShift - m0);
                    uint64_t sum[2] = {0, 0};
                    auto weigh32 = [&](const uint32_t *v, int k) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            unpair(fma2(pair(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, m2), x0, x1);
                            const float p0 = exp2_sfu(x0), p1 = exp2_sfu(x1);
                            sum[e & 1] = add2(sum[e & 1], pair(p0, p1));
                            pk[e] = TcType<T>::pack(p0, p1);
                        }
                        tc_st16(tm_s + kTmemP + 16 * k, pk);
                    };
                    if (plain) {
                        tc_ld32(tm_s, s0);
                        weigh32(s1, 3);
                        tc_loaded(s0);
                        tc_ld32(tm_s + 32, s1);
                        weigh32(s2, 2);
                        tc_loaded(s1);
                        weigh32(s1, 1);
                        weigh32(s0, 0);
                    } else {
#pragma unroll 1
                        for (int k = nch - 1; k >= 0; --k) {
                            const uint32_t w = seen32(tl.nodes, bits, lim, k);
                            if (!__any_sync(0xFFFFFFFFu, real && w != 0)) {
                                uint32_t none[16] = {};
                                tc_st16(tm_s + kTmemP + 16 * k, none);
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
                    ok = wait(&s.pv_done[0], (i - 1) & 1);
                    if (!ok)
                        break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.p_full[x]);
            }
            if (!ok)
                break;
            const bool whole = u.n_parts == 1;
            float *slot = whole ? nullptr : part_slot<Sh::kRows>(a, blockIdx.x, u.part);
            if (end > u.tile) {
                ok = wait(&s.pv_done[t], NT == 1 ? (i - 1) & 1 : n_done & 1);
                if (!ok)
                    break;
                ++n_done;
                tc_fence_after();
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                const uint32_t *odd = s.odd[n % kGuardRing];
                const uint32_t any_odd = *reinterpret_cast<const volatile uint32_t *>(odd + 12);
                T *dst = real ? reinterpret_cast<T *>(a.out) + row_place(a, u, ur) : nullptr;
                if (busy) {
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t o[32];
                        tc_load(tm_o + 32 * k, o);
                        if (any_odd && real) {
                            uint32_t x[32];  // rare; the call keeps only this copy in memory
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[e] = o[e];
                            put_back32<T, PROMPT>(a, u, odd, tok, 32 * k, x);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = x[e];
                        }
                        if (real) {
                            if (whole) {
                                store_row32<T>(dst + 32 * k, o, inv);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    __stcg(reinterpret_cast<uint4 *>(slot + part_quad<Sh::kRows>(8 * k + e / 4, ur)),
                                           make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                            }
                        }
                    }
                    if (real && !whole) {
                        __stcg(slot + (size_t)Sh::kRows * D + ur, m);
                        __stcg(slot + (size_t)Sh::kRows * D + Sh::kRows + ur, l);
                    }
                }
                tc_fence_before();
            }
            if (!whole) {
                __threadfence();
                mbar_arrive(&s.joined);
                ok = wait(&s.joined, n_join++ & 1);
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
                ok = wait(&s.joined, n_join++ & 1);
                if (!ok)
                    break;
                if (s.last) {
                    __threadfence();
                    ok = join_parts<T, Sh::kRows>(a, u, tid, Sh::kSoftmax, [&] {
                        __threadfence();
                        mbar_arrive(&s.joined);
                        return wait(&s.joined, n_join++ & 1);
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
        if (warp == kLoadWarp && lane == 0) {
            await_copies<ST>(s.kv_full, s.asked_kv);
            await_copies<Sh::kQBuf>(s.q_full, s.asked_q);
        }
        if (warp == kMmaWarp) {
            await_products(&s.settled);
            give_up(a);
        }
    }
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
namespace {

template <typename T, int D, int NT, bool PROMPT>
cudaError_t launch_tc(const AttendArgs &a, cudaStream_t st)
{
    using Sh = TcShape<D, NT>;
    TcMaps maps;
    TcBoxes box;
    if (!tc_make_maps(a, TcType<T>::kFmt == 1, kKeys, &maps, &box))
        return cudaErrorInvalidValue;
    const long long tokens = PROMPT ? a.seq.M : (long long)a.seq.B * a.seq.T;
    const cudaError_t err = cudaFuncSetAttribute(attend_tc_kernel<T, D, NT, PROMPT>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (err != cudaSuccess)
        return err;
    dim3 grid(kAttendCtas);
    if (PROMPT)
        grid = dim3((unsigned)(tokens / (NT * box.tok_tile) + a.seq.B), (unsigned)a.cache.H);
    attend_tc_kernel<T, D, NT, PROMPT><<<grid, Sh::kThreads, Sh::kSmem, st>>>(a, maps, box);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_tc_d(const AttendArgs &a, cudaStream_t st)
{
    if (a.seq.cu)
        return launch_tc<T, D, 2, true>(a, st);
    return a.seq.T * a.G <= kKeys ? launch_tc<T, D, 1, false>(a, st) : launch_tc<T, D, 2, false>(a, st);
}

}  // namespace

// Whether the tensor-core kernel takes the call: 16-bit elements, a head size
// it has tiles for, a key head's query heads within one tile, TMA's alignment.
bool attend_tc_takes(const AttendArgs &a, spec_dtype dt)
{
    if (dt == SPEC_F32 || (a.cache.D != 64 && a.cache.D != 128) || a.G > kKeys)
        return false;
    if (a.seq.cu && a.seq.M == 0)
        return false;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.out) |
                         reinterpret_cast<uintptr_t>(a.cache.kv) | reinterpret_cast<uintptr_t>(a.staged);
    return at % 16 == 0 && tc_available();
}

cudaError_t launch_attend_tc(const AttendArgs &a, spec_dtype dt, cudaStream_t st)
{
    // Small units two to an SM, or large ones with two chains each?  Rounds: small
    // up to 64 rows a key head (decoding at batch 32 41 us, 47 with one large
    // unit an SM); up to 128 rows take one query tile of attend_tc_kernel (72
    // rows, 32 sequences: 70 us, 84 with two; 126 rows, 8 sequences: 47 and 47).
    // Prompts: small up to kShortPrompt tokens a sequence on average, where a
    // unit's start and end cost more than its tiles (mean 158 tokens: 22.5 us
    // against 28.7; 200: 32.8, 36.9; 512: equal; 1200: 139, 135; 2000: 295, 276).
    // The mean is all that the host knows: one prompt of 14000 tokens beside 30 of
    // 60 would take 1059 us in large units (here 1210), 8 pieces of 512 on 8000
    // cached keys 418 (465), one of 512 on 16000 the same.
    if (a.seq.cu) {
        if (a.seq.M <= (long long)kShortPrompt * a.seq.B)
            return launch_attend_few(a, dt, st);
    } else if (a.seq.T * a.G <= 64) {
        return launch_attend_few(a, dt, st);
    }
    if (a.cache.D == 64)
        return dt == SPEC_BF16 ? launch_tc_d<__nv_bfloat16, 64>(a, st) : launch_tc_d<__half, 64>(a, st);
    return dt == SPEC_BF16 ? launch_tc_d<__nv_bfloat16, 128>(a, st) : launch_tc_d<__half, 128>(a, st);
}

size_t attend_tc_workspace(int T, int Hq, int H, int D)
{
    const long long rows = (long long)T * (Hq / (H > 0 ? H : 1));
    const size_t part = rows <= kKeys ? part_floats<128>(D) : part_floats<256>(D);
    const size_t tc = align256(kPartHead + 2 * kAttendCtas * part * sizeof(float)), few = attend_few_workspace(D);
    return tc > few ? tc : few;
}

}  // namespace spec
