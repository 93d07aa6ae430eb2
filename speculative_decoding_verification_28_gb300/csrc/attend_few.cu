// attend_few.cu -- attention on the tensor cores in small units: rounds where a
// key head has few query rows (up to 64: decoding and short chains), and
// short prompts (128 rows a unit, where attend_tc.cu's have 256).
//
// The mathematics and the softmax are attend_tc.cu's; the split is made for a
// bandwidth-bound stream.  A tile of 128 keys arrives every 3000 cycles an SM
// (512 bytes a key of 128 columns, HBM), its chain of score, softmax and
// product takes about as long, and a unit's start and end as long again.  So
// two CTAs share an SM, each with one buffer of everything (TMEM: 128 columns
// of scores and weights, 128 of O; a ring of two or three tiles), and one's
// chain runs while the other's keys arrive.  Measured: 256 chains of 9 tokens,
// 32 / 8 heads of 128 over 2.3 GB of keys, 378 us (6.0 TB/s, 0.89 of a copy);
// 64 of them 129 us (4.5 TB/s); decoding at batch 32 over 109 MB 41 us with a
// cold cache, of which 6 pass before the first tile is there and 4 in joins;
// 8 prompts of 158 tokens on average 22 us, all of it latency.  The weights are
// rounded to the storage type as in attend_tc.cu.
#include "tcgen.cuh"

namespace spec {

constexpr int kFewRows = 64;        // most query rows of a round's unit
constexpr int kFewPromptRows = 128; // and of a prompt's
constexpr int kFewCtas = 2 * kAttendCtas;
constexpr int kFewThreads = 192;
constexpr int kFewTmemP = 64;  // columns of the scores where the weights begin

template <int D, bool PROMPT>
struct FewShape {
    static constexpr int kRows = PROMPT ? kFewPromptRows : kFewRows;
    static constexpr int kPanels = D / 64;
    static constexpr int kPanel = kKeys * 128;
    static constexpr int kTile = kPanels * kPanel;       // bytes of a K or V tile
    static constexpr int kQPanel = kRows * 128;          // the product reads 128 rows: what follows
    static constexpr int kQ = kPanels * kQPanel;
    static constexpr int kStages = D == 128 ? (PROMPT ? 2 : 3) : 5;
};
template <int STAGES>
struct FewShared {
    uint64_t kv_full[STAGES], kv_empty[STAGES];
    uint64_t q_full, q_empty, s_full, p_full, pv_done, joined, settled;
    uint32_t asked_kv, asked_q;  // copies that the load warp asked for in all
    uint32_t scan[8];
    Run run;
    uint32_t tmem;
    int abort, last;
    uint32_t odd[kGuardRing][13];
};
template <int D, bool PROMPT>
constexpr int few_smem()
{
    using Sh = FewShape<D, PROMPT>;
    return Sh::kStages * Sh::kTile + Sh::kQ + (int)sizeof(FewShared<Sh::kStages>);
}
static_assert(few_smem<128, false>() <= 115712 && few_smem<64, false>() <= 115712, "two CTAs an SM");
static_assert(few_smem<128, true>() <= 115712 && few_smem<64, true>() <= 115712, "two CTAs an SM");

template <typename T, int D, bool PROMPT>
__global__ void __launch_bounds__(kFewThreads, 2)
    attend_few_kernel(const AttendArgs a, const __grid_constant__ TcMaps maps, const TcBoxes box)
{
    using Sh = FewShape<D, PROMPT>;
    constexpr int ST = Sh::kStages;
    extern __shared__ __align__(1024) unsigned char base[];
    unsigned char *ring_p = base + Sh::kQ;  // queries first: rows past theirs are read from the ring
    FewShared<ST> &s = *reinterpret_cast<FewShared<ST> *>(ring_p + ST * Sh::kTile);
    const uint32_t q_smem = smem_addr(base), ring = smem_addr(ring_p);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Shape sh{kKeys, box.tok_tile * a.G, a.G};
    constexpr int kMmaWarp = 4, kLoadWarp = 5;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&s.kv_full[i], 1);
            mbar_init(&s.kv_empty[i], 1);
        }
        mbar_init(&s.q_full, 1);
        mbar_init(&s.q_empty, 1);
        mbar_init(&s.s_full, 1);
        mbar_init(&s.p_full, 4);
        mbar_init(&s.pv_done, 1);
        mbar_init(&s.joined, 4);
        mbar_init(&s.settled, 1);
        fence_mbar_init();
        s.abort = 0;
        s.run.begin = s.run.end = 0;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_addr(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (warp == kLoadWarp && lane < 3) {
        const CUtensorMap *m = lane == 0 ? &maps.q : lane == 1 ? &maps.kv : &maps.node;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    AttendUnit first{};
    bool some = true;
    if (PROMPT) {
        some = prompt_unit(a, sh, first);
    } else {
        __syncthreads();  // run.begin / end above come before find_run's
        find_run<kFewThreads>(a, sh, s.scan, &s.run);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem, tm_o = tmem + 128;

    const long long limit = a.wait_clocks;  // by itself: the waits' reference to all of `a` would put it on the stack
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, &s.abort, limit));
    };
    Units<PROMPT> units(a, sh, s.run, first, some);
    AttendUnit u{};

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            uint32_t it = 0, n = 0;
            bool ok = true;
            while (ok && units.next(u)) {
                // the first keys before the queries: those wait for the unit
                // before to be scored
                for (int tile = u.tile; ok && tile < u.tile_end; ++tile) {
                    const KvBox k = kv_box<Sh::kPanels>(a, maps, box, u, tile, !PROMPT && tile == u.n_tiles - 1);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int sg = it % ST;
                        ok = ok && wait_phase(&s.kv_empty[sg], ((it / ST) & 1) ^ 1, &s.abort, limit);
                        if (!ok)
                            break;
                        mbar_arrive_expect_tx(&s.kv_full[sg], k.bytes);
#pragma unroll
                        for (int p = 0; p < Sh::kPanels; ++p)
                            tma_load_3d(ring + sg * Sh::kTile + p * Sh::kPanel, k.m, p * 64, k.y, k.z + kv * k.zv,
                                        &s.kv_full[sg]);
                        ++it;
                        if (tile == u.tile && kv == 0) {
                            ok = wait_phase(&s.q_empty, (n & 1) ^ 1, &s.abort, limit);
                            if (!ok)
                                break;
                            mbar_arrive_expect_tx(&s.q_full, Sh::kPanels * box.q_tok * a.G * 128);
#pragma unroll
                            for (int p = 0; p < Sh::kPanels; ++p)
                                tma_load_4d(q_smem + p * Sh::kQPanel, &maps.q, p * 64, 0, u.h,
                                            (int)u.seq.tok0 + u.row0 / a.G, &s.q_full);
                            ++n;
                        }
                    }
                }
            }
            s.asked_kv = it;
            s.asked_q = n;
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------- mma and guard
        const uint32_t one = elect_one();
        const uint32_t ideo = tc_idesc<T>(D, true);
        auto commit = [&](uint64_t *bar) {
            if (one)
                tc_commit(bar);
        };
        uint32_t i = 0, n = 0;  // tiles, units
        bool ok = true;
        while (ok && units.next(u)) {
            uint32_t *odd = s.odd[n % kGuardRing];
            if (lane < 13)
                odd[lane] = 0;
            __syncwarp();
            int g = 0;
            for (int tile = u.tile; ok && tile < u.tile_end; ++tile, ++i) {
                const uint32_t sk = (2 * i) % ST, sv = (2 * i + 1) % ST;
                const Tile tl = tile_of<PROMPT>(u, tile);
                if (tile == u.tile)
                    ok = wait(&s.q_full, n & 1);
                ok = ok && wait(&s.kv_full[sk], ((2 * i) / ST) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t qd = operand(q_smem, 16), kd = operand(ring + sk * Sh::kTile, 16);
                const uint32_t ides = tc_idesc<T>(min(kKeys, (tl.valid + 15) & ~15), false);
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    mma_ss(one, tmem, qd + (((c / 4) * Sh::kQPanel + (c % 4) * 32) >> 4),
                           kd + (((c / 4) * Sh::kPanel + (c % 4) * 32) >> 4), ides, c > 0);
                commit(&s.s_full);
                commit(&s.kv_empty[sk]);
                if (tile + 1 == u.tile_end)
                    commit(&s.q_empty);
                ok = wait(&s.kv_full[sv], ((2 * i + 1) / ST) & 1);
                if (ok && guarded(tl))
                    guard_tile<T, Sh::kPanels>(ring_p + sv * Sh::kTile, tl, odd, g);
                ok = ok && wait(&s.p_full, i & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t vd = operand(ring + sv * Sh::kTile, Sh::kPanel), pt = tmem + kFewTmemP;
                mma_ts(one, tm_o, pt, vd, ideo, tile > u.tile);
                if (tl.valid > kKeys - 16) {
#pragma unroll
                    for (int c = 1; c < kKeys / 16; ++c)
                        mma_ts(one, tm_o, pt + c * 8, vd + c * (2048 >> 4), ideo, 1);
                } else {
                    for (int c = 1; c < (tl.valid + 15) / 16; ++c)
                        mma_ts(one, tm_o, pt + c * 8, vd + c * (2048 >> 4), ideo, 1);
                }
                commit(&s.kv_empty[sv]);
                if (tile + 1 == u.tile_end)
                    commit(&s.pv_done);
            }
            ++n;
        }
    } else {
        // ---------------------------------------------------------- softmax
        if (!PROMPT && blockIdx.x == 0 && warp == 0)
            flag_if_gave_up(a);
        const int r = tid;  // row of the unit = TMEM lane
        const uint32_t lanes = (uint32_t)warp << 21, tm_s = tmem + lanes;
        const float c = a.scale_log2;
        const uint64_t c2 = pair(c, c);
        uint32_t i = 0, n = 0, joins = 0;
        bool ok = true;
        while (ok && units.next(u)) {
            const bool real = r < u.n_rows;
            const bool busy = __any_sync(0xFFFFFFFFu, real);
            const int tok = (u.row0 + r) / a.G;
            uint64_t bits = 0;  // nodes that the row sees
            if (!PROMPT && real && u.tile_end == u.n_tiles) {
                bits = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
                if (u.seq.n < 64)
                    bits &= (1ull << u.seq.n) - 1;
            }
            float m = -INFINITY, l = 0.0f;
            for (int tile = u.tile; tile < u.tile_end; ++tile, ++i) {
                ok = wait(&s.s_full, i & 1);
                if (!ok)
                    break;
                tc_fence_after();
                if (busy) {
                    const Tile tl = tile_of<PROMPT>(u, tile);
                    const int nch = (tl.valid + 31) / 32;
                    uint32_t s0[32], s1[32];
                    const int lim = PROMPT ? min(tl.valid, u.seq.prefix + tok + 1 - tile * kKeys) : tl.valid;
                    const bool plain = !tl.nodes && !__any_sync(0xFFFFFFFFu, lim < kKeys);
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
                    if (tile == u.tile) {
                        m = mx;
                    } else if (__any_sync(0xFFFFFFFFu, mx > m + TcType<T>::kLazy)) {
                        // O is at rest: these scores came after its last product
                        float f = 1.0f;
                        if (mx > m + TcType<T>::kLazy) {
                            f = exp2_sfu(m - mx);  // 0 when nothing was seen before
                            m = mx;
                        }
                        l *= f;
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[16];
                            tc_ld16(tm_o + lanes + k, o);
                            tc_wait_ld();
                            tc_pin<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st16(tm_o + lanes + k, o);
                        }
                    }
                    const float m0 = m == -INFINITY ? 0.0f : m;
                    const uint64_t m2 = pair(TcType<T>::kShift - m0, TcType<T>::kShift - m0);
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
                            pk[e] = TcType<T>::pack(p0, p1);
                        }
                        tc_st16(tm_s + kFewTmemP + 16 * k, pk);
                    };
                    if (plain) {
                        weigh32(s1, 3);
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
                                tc_st16(tm_s + kFewTmemP + 16 * k, none);
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
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.p_full);
            }
            ok = ok && wait(&s.pv_done, n & 1);
            if (!ok)
                break;
            tc_fence_after();
            const bool whole = u.n_parts == 1;
            float *slot = whole ? nullptr : part_slot<Sh::kRows>(a, blockIdx.x, u.part);
            if (busy) {
                const float f = !whole ? 1.0f : l > 0.0f || l != l ? 1.0f / l : 0.0f;
                const uint32_t *odd = s.odd[n % kGuardRing];
                const uint32_t any_odd = *reinterpret_cast<const volatile uint32_t *>(odd + 12);
                T *dst = real ? reinterpret_cast<T *>(a.out) + row_place(a, u, r) : nullptr;
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    uint32_t o[32];
                    tc_load(tm_o + lanes + k, o);
                    if (any_odd && real) {
                        uint32_t x[32];  // rare; the call keeps only this copy in memory
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = o[e];
                        put_back32<T, PROMPT>(a, u, odd, tok, k, x);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = x[e];
                    }
                    if (!real)
                        continue;
                    if (whole) {
                        store_row32<T>(dst + k, o, f);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            __stcg(reinterpret_cast<uint4 *>(slot + part_quad<Sh::kRows>((k + e) / 4, r)),
                                   make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                    }
                }
                if (real && !whole) {
                    __stcg(slot + (size_t)Sh::kRows * D + r, m);
                    __stcg(slot + (size_t)Sh::kRows * D + Sh::kRows + r, l);
                }
            }
            tc_fence_before();
            if (!whole) {
                __threadfence();
                __syncwarp();
                if (lane == 0)
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
                if (lane == 0)
                    mbar_arrive(&s.joined);
                ok = wait(&s.joined, joins++ & 1);
                if (!ok)
                    break;
                if (s.last) {
                    __threadfence();
                    ok = join_parts<T, Sh::kRows>(a, u, tid, 128, [&] {
                        __threadfence();
                        __syncwarp();
                        if (lane == 0)
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
        if (warp == kLoadWarp && lane == 0) {
            await_copies<ST>(s.kv_full, s.asked_kv);
            await_copies<1>(&s.q_full, s.asked_q);
        }
        if (warp == kMmaWarp) {
            await_products(&s.settled);
            give_up(a);
        }
    }
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
}

namespace {

template <typename T, int D, bool PROMPT>
cudaError_t launch_few(const AttendArgs &a, cudaStream_t st)
{
    using Sh = FewShape<D, PROMPT>;
    TcMaps maps;
    TcBoxes box;
    if (!tc_make_maps(a, TcType<T>::kFmt == 1, Sh::kRows, &maps, &box))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(attend_few_kernel<T, D, PROMPT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem<D, PROMPT>());
    if (e != cudaSuccess)
        return e;
    dim3 grid(kFewCtas);
    if (PROMPT)
        grid = dim3((unsigned)(a.seq.M / box.tok_tile + a.seq.B), (unsigned)a.cache.H);
    attend_few_kernel<T, D, PROMPT><<<grid, kFewThreads, few_smem<D, PROMPT>(), st>>>(a, maps, box);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_few_t(const AttendArgs &a, cudaStream_t st)
{
    if (a.cache.D == 64)
        return a.seq.cu ? launch_few<T, 64, true>(a, st) : launch_few<T, 64, false>(a, st);
    return a.seq.cu ? launch_few<T, 128, true>(a, st) : launch_few<T, 128, false>(a, st);
}

}  // namespace

cudaError_t launch_attend_few(const AttendArgs &a, spec_dtype dt, cudaStream_t st)
{
    return dt == SPEC_BF16 ? launch_few_t<__nv_bfloat16>(a, st) : launch_few_t<__half>(a, st);
}

size_t attend_few_workspace(int D)
{
    return align256(kPartHead + 2 * kFewCtas * part_floats<kFewRows>(D) * sizeof(float));
}

}  // namespace spec
