// attend_tc.cu -- attention on the tensor cores (tcgen05), for bf16 and fp16
// caches with heads of 64 or 128.
//
//   S = Q K^T in TMEM;  P = 2^(c S - m) in TMEM, rounded to the storage type;
//   O += P V in TMEM, fp32
//
// with one pass over the keys.  A row's m is a running maximum that is only
// moved when a tile's maximum is more than 2^8 above it: O and the sum are
// then rescaled.  Between moves the weights exceed 1 by at most 2^8, which
// fp32 sums and bf16 / fp16 weights hold without loss of precision.
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
// tensor pipe.
#include <cuda.h>

#include "attend_common.cuh"
#include "bulk_copy.cuh"
#include "verify_common.cuh"

namespace spec {

constexpr int kKeys = 128;  // keys of a tile, rows of a query tile
constexpr int kTcWaitLimit = 2000;  // probes of up to ~1 ms, after a wait that gave up
constexpr long long kTcWaitClocks = 4000000000ll;  // about 2 s
constexpr float kLazy = 8.0f;       // base-2 headroom of the running maximum
constexpr int kGuardRing = 8;       // units whose guard words may be live at once

// ---------------------------------------------------------------------------
// inline PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
                 "[%5];" ::"r"(dst),
                 "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int w, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
                 "%5}], [%6];" ::"r"(dst),
                 "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
                 : "memory");
}
// one probe of a phase, without a time of its own to sleep: it wakes sooner
__device__ __forceinline__ bool mbar_poll(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// keeps what is done with loaded registers behind the wait for them
template <int N>
__device__ __forceinline__ void tc_pin(uint32_t *r)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand with 128-byte swizzle: rows of 128 bytes, groups of
// eight rows 1024 bytes apart, panels of 64 elements `panel` bytes apart
// (used by operands whose long axis is not the summed one).
// Operand descriptors: the upper word is the same for all, the lower holds
// the address and the panel step.  Only the elected lane issues (`one`), but
// the whole warp computes, so that the words stay in uniform registers: built
// per lane they cost more than the 64 cycles of a 128 x 128 x 16 product.
constexpr uint32_t kOperandHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t panel) { return (addr >> 4) | ((panel >> 4) << 16); }

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

// D = A B (+ D): A and B in shared memory
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(one), "n"(kOperandHi)
                 : "memory");
}
// A in TMEM
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "mov.b64 y, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(one), "n"(kOperandHi)
                 : "memory");
}

#define SPEC_R4(x, i) x[i], x[i + 1], x[i + 2], x[i + 3]
#define SPEC_OUT4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define SPEC_IN4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])

// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : SPEC_OUT4(r, 0), SPEC_OUT4(r, 4), SPEC_OUT4(r, 8), SPEC_OUT4(r, 12), SPEC_OUT4(r, 16),
                   SPEC_OUT4(r, 20), SPEC_OUT4(r, 24), SPEC_OUT4(r, 28)
                 : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
                     SPEC_IN4(r, 0),
                 SPEC_IN4(r, 4), SPEC_IN4(r, 8), SPEC_IN4(r, 12), SPEC_IN4(r, 16), SPEC_IN4(r, 20), SPEC_IN4(r, 24),
                 SPEC_IN4(r, 28), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15};" ::SPEC_IN4(r, 0),
                 SPEC_IN4(r, 4), SPEC_IN4(r, 8), SPEC_IN4(r, 12), "r"(addr)
                 : "memory");
}

// the loads so far have arrived; r are registers of theirs
__device__ __forceinline__ void tc_loaded(uint32_t *r)
{
    tc_wait_ld();
    tc_pin<32>(r);
}
__device__ __forceinline__ void tc_load(uint32_t addr, uint32_t *r)
{
    tc_ld32(addr, r);
    tc_loaded(r);
}

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float max32(const uint32_t *r)
{
    float m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t *x = r + 16 * h;
        m[h] = __uint_as_float(x[15]);
#pragma unroll
        for (int e = 0; e < 14; e += 2)
            m[h] = max3(m[h], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        m[h] = fmaxf(m[h], __uint_as_float(x[14]));
    }
    return fmaxf(m[0], m[1]);
}

template <typename T>
struct TcType;
template <>
struct TcType<__nv_bfloat16> {
    static constexpr uint32_t kFmt = 1;
    __device__ static uint32_t pack(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    // exponent of all ones in either half
    __device__ static bool odd(uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }
    __device__ static uint32_t max_abs(uint32_t m, uint32_t w) { return max_nan_bf16x2(m, w & 0x7FFF7FFFu); }
    static constexpr uint32_t kExp = 0x7F80u;
};
template <>
struct TcType<__half> {
    static constexpr uint32_t kFmt = 0;
    __device__ static uint32_t pack(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static bool odd(uint32_t w) { return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u; }
    __device__ static uint32_t max_abs(uint32_t m, uint32_t w) { return max_nan_f16x2(m, w & 0x7FFF7FFFu); }
    static constexpr uint32_t kExp = 0x7C00u;
};

// instruction descriptor: fp32 accumulators, both operands T, M = 128
template <typename T>
__device__ __forceinline__ uint32_t tc_idesc(int n, bool b_rows_summed)
{
    return (1u << 4) | (TcType<T>::kFmt << 7) | (TcType<T>::kFmt << 10) | ((b_rows_summed ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// ---------------------------------------------------------------------------
// shapes
// ---------------------------------------------------------------------------
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
    static constexpr int kThreads = kSoftmax + 96;
    static constexpr int kRows = 128 * NT;
    static constexpr uint32_t kTmemO = 256;
};

struct TcMaps {
    CUtensorMap q, kv, node;
};
// rows the maps' boxes bring
struct TcBoxes {
    int q_tok, tok_tile, kv_rows, node_rows;
};

template <int STAGES>
struct TcShared {
    uint64_t kv_full[STAGES], kv_empty[STAGES], q_full[2], q_empty[2];
    uint64_t v_ok[STAGES];  // guarded tiles: a stage's next one waits for its own consumption
    uint64_t s_full[2], p_full[2], pv_done[2], joined;
    long long scan[16];
    Run run;
    uint32_t tmem;
    int abort, last;
    uint32_t odd[kGuardRing][12];  // keys of the guarded tiles with a value that is not finite
};

// A tile of a unit: how many of its keys are real, and whether some row does
// not see all of those.
struct Tile {
    int valid;
    bool nodes, masked;
};
template <bool PROMPT>
__device__ __forceinline__ Tile tile_of(const AttendUnit &u, int tile)
{
    Tile t;
    if (PROMPT) {
        t.nodes = false;
        t.valid = min(kKeys, u.seen_last - tile * kKeys);
        t.masked = (tile + 1) * kKeys > u.seen_first;
    } else {
        t.nodes = tile == u.n_tiles - 1;
        t.valid = t.nodes ? u.seq.n : min(kKeys, u.seq.prefix - tile * kKeys);
        t.masked = t.nodes;
    }
    return t;
}
__device__ __forceinline__ bool guarded(const Tile &t) { return t.masked || (t.valid & 15); }

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

// Walks the units of a CTA: a prompt's one, or a round's run.
template <bool PROMPT>
struct Units {
    UnitWalk walk;
    AttendUnit one;
    bool fresh;
    __device__ Units(const AttendArgs &a, const Shape &sh, const Run &r, const AttendUnit &u) : walk(a, sh, r), one(u), fresh(true)
    {
    }
    __device__ bool next(AttendUnit &u)
    {
        if (!PROMPT)
            return walk.next(u);
        u = one;
        const bool was = fresh;
        fresh = false;
        return was;
    }
};

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
    auto wait1 = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (mbar_poll(bar, parity))
            return true;
        const long long t0 = clock64();
        while (!mbar_poll(bar, parity)) {
            if (*reinterpret_cast<volatile int *>(&s.abort))
                return false;
            if (clock64() - t0 > kTcWaitClocks) {
                *reinterpret_cast<volatile int *>(&s.abort) = 1;
                return false;
            }
        }
        return true;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, wait1(bar, parity));
    };
    Units<PROMPT> units(a, sh, s.run, first);
    AttendUnit u{};

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            const int heads = a.cache.N * a.cache.H;  // V slabs follow the K slabs
            uint32_t it = 0, n = 0;
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
                for (int tile = u.tile; ok && tile < u.tile_end; ++tile) {
                    const bool nodes = !PROMPT && tile == u.n_tiles - 1;
                    const CUtensorMap *m = nodes ? &maps.node : &maps.kv;
                    const bool st = nodes && a.seq.staged;
                    const int y = st ? 0 : u.seq.slot0 + (nodes ? u.seq.prefix : tile * kKeys);
                    const int z = st ? u.b * a.cache.H + u.h : u.seq.row * a.cache.H + u.h;
                    const int zv = st ? a.seq.B * a.cache.H : heads;
                    const uint32_t bytes = Sh::kPanels * 128 * (nodes ? box.node_rows : box.kv_rows);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int sg = it % ST;
                        ok = ok && wait1(&s.kv_empty[sg], ((it / ST) & 1) ^ 1);
                        if (!ok)
                            break;
                        mbar_arrive_expect_tx(&s.kv_full[sg], bytes);
#pragma unroll
                        for (int p = 0; p < Sh::kPanels; ++p)
                            tma_load_3d(ring + sg * Sh::kTile + p * Sh::kPanel, m, p * 64, y, z + kv * zv, &s.kv_full[sg]);
                        ++it;
                    }
                }
                ++n;
            }
            if (!ok) {
                // after a wait that gave up: the copies in flight land first
                for (uint32_t i = it > ST ? it - ST : 0; i < it; ++i)
                    for (int k = 0; k < kTcWaitLimit && !mbar_try_wait(&s.kv_full[i % ST], (i / ST) & 1); ++k)
                        ;
                for (uint32_t i = n > 0 ? n - 1 : 0; i <= n; ++i)
                    for (int k = 0; k < kTcWaitLimit && !mbar_try_wait(&s.q_full[i % Sh::kQBuf], (i / Sh::kQBuf) & 1); ++k)
                        if (i == n && k > 8)
                            break;  // unit n's queries may not have been asked for
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------------- mma
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
            Units<PROMPT> ahead(a, sh, s.run, first);
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
    } else if (warp == kLoadWarp + 1) {
        // ------------------------------------------------------------ guard
        uint32_t i = 0, n = 0;
        bool ok = true;
        while (ok && units.next(u)) {
            uint32_t *odd = s.odd[n % kGuardRing];
            if (lane < 12)
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
                unsigned char *v = ring_p + sg * Sh::kTile;
                for (int r = tl.valid + (lane >> 3); r < ((tl.valid + 15) & ~15); r += 4)
#pragma unroll
                    for (int p = 0; p < Sh::kPanels; ++p)
                        *reinterpret_cast<uint4 *>(v + p * Sh::kPanel + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                if (tl.masked) {
                    uint32_t m = 0;
                    for (int r = lane >> 3; r < tl.valid; r += 4)
#pragma unroll
                        for (int p = 0; p < Sh::kPanels; ++p) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(v + p * Sh::kPanel + r * 128 + (lane & 7) * 16);
                            m = TcType<T>::max_abs(TcType<T>::max_abs(m, x.x), x.y);
                            m = TcType<T>::max_abs(TcType<T>::max_abs(m, x.z), x.w);
                        }
                    if (__any_sync(0xFFFFFFFFu, TcType<T>::odd(m))) {
                        // rare: take the values out, remember their keys
                        for (int r = lane >> 3; r < tl.valid; r += 4) {
                            for (int p = 0; p < Sh::kPanels; ++p) {
                                uint32_t *w = reinterpret_cast<uint32_t *>(v + p * Sh::kPanel + r * 128 + (lane & 7) * 16);
                                for (int e = 0; e < 4; ++e) {
                                    uint32_t x = w[e];
                                    if (!TcType<T>::odd(x))
                                        continue;
                                    if ((x & TcType<T>::kExp) == TcType<T>::kExp)
                                        x &= 0xFFFF0000u;
                                    if ((x >> 16 & TcType<T>::kExp) == TcType<T>::kExp)
                                        x &= 0x0000FFFFu;
                                    w[e] = x;
                                    atomicOr(&odd[g * 4 + (r >> 5)], 1u << (r & 31));
                                }
                            }
                        }
                    }
                    ++g;
                }
                __threadfence_block();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.v_ok[sg]);
                    mbar_arrive(&s.kv_empty[sg]);
                }
            }
            ++n;
        }
    } else {
        // ---------------------------------------------------------- softmax
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
                    uint64_t bits = 0;
                    const int nch = (tl.valid + 31) / 32;
                    auto masked = [&](uint32_t *v, int k) {
                        if (tl.nodes) {
                            const uint32_t w = (uint32_t)(bits >> (32 * k));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(w >> e & 1))
                                    v[e] = 0xFF800000u;
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * k + e >= lim)
                                    v[e] = 0xFF800000u;
                        }
                    };
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
#pragma unroll 1
                        for (int k = 0; k < nch; ++k) {
                            tc_load(tm_s + 32 * k, s0);
                            masked(s0, k);
                            mx = fmaxf(mx, max32(s0));
                        }
                    }
                    mx *= c;
                    float f = 1.0f;
                    if (tile == u.tile) {
                        m = mx;
                    } else if (__any_sync(0xFFFFFFFFu, mx > m + kLazy)) {
                        if (mx > m + kLazy) {
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
                    const uint64_t c2 = pair(c, c), m2 = pair(-m0, -m0);
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
                            tc_load(tm_s + 32 * k, s0);
                            masked(s0, k);
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
                uint32_t any_odd = 0;
#pragma unroll
                for (int k = 0; k < 12; ++k)
                    any_odd |= *reinterpret_cast<const volatile uint32_t *>(odd + k);
                T *dst = real ? reinterpret_cast<T *>(a.out) + row_place(a, u, ur) : nullptr;
                if (busy) {
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t o[32];
                        tc_load(tm_o + 32 * k, o);
                        if (any_odd && real) {
                            // the values taken out of V go where they are seen
                            int g = 0;
                            for (int tile = u.tile; tile < u.tile_end; ++tile) {
                                const Tile tl = tile_of<PROMPT>(u, tile);
                                if (!tl.masked)
                                    continue;
                                for (int key = 0; key < tl.valid; ++key) {
                                    if (!(odd[g * 4 + (key >> 5)] >> (key & 31) & 1))
                                        continue;
                                    bool sees;
                                    const T *v;
                                    if (tl.nodes) {
                                        const uint64_t bits =
                                            a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
                                        sees = bits >> key & 1;
                                    } else {
                                        sees = tile * kKeys + key <= u.seq.prefix + tok;
                                    }
                                    if (tl.nodes && a.seq.staged)
                                        v = reinterpret_cast<const T *>(a.staged) +
                                            ((a.st_v + (long long)u.b * a.cache.H + u.h) * a.seq.T + key) * D;
                                    else
                                        v = reinterpret_cast<const T *>(a.cache.kv) +
                                            ((a.cache.v_slab + (long long)u.seq.row * a.cache.H + u.h) * a.cache.S +
                                             u.seq.slot0 + (tl.nodes ? u.seq.prefix : tile * kKeys) + key) *
                                                D;
                                    if (sees)
#pragma unroll
                                        for (int e = 0; e < 32; ++e) {
                                            const float f = Storage<T>::at(v, 32 * k + e);
                                            if (!(fabsf(f) <= 3.0e38f))
                                                o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
                                        }
                                }
                                ++g;
                            }
                        }
                        if (real) {
                            if (whole) {
#pragma unroll
                                for (int e = 0; e < 32; e += 8) {
                                    uint4 w;
                                    w.x = TcType<T>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                                    w.y = TcType<T>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                                    w.z = TcType<T>::pack(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                                    w.w = TcType<T>::pack(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                                    *reinterpret_cast<uint4 *>(dst + 32 * k + e) = w;
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    __stcg(reinterpret_cast<uint4 *>(slot + (size_t)ur * D + 32 * k + e),
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
                    join_parts<T, Sh::kRows>(a, u, warp, Sh::kSoftmax / 32);
                }
            }
            ++n;
        }
    }
    if (*reinterpret_cast<volatile int *>(&s.abort) && lane == 0 && a.flags && u.seq.ok)
        atomicOr(a.flags + u.b, SPEC_FLAG_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// 16-bit elements, innermost extent D in panels of 64, the further extents,
// strides (bytes) and box as given
bool make_map(CUtensorMap *m, bool bf16, const void *p, int rank, const cuuint64_t *dim, const cuuint64_t *stride,
              const cuuint32_t *box)
{
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return encode_tiled()(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
                          const_cast<void *>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int NT, bool PROMPT>
cudaError_t launch_tc(const AttendArgs &a, cudaStream_t st)
{
    using Sh = TcShape<D, NT>;
    const bool bf16 = TcType<T>::kFmt == 1;
    const cuuint64_t e = 2, row = (cuuint64_t)D * e;
    const long long tokens = PROMPT ? a.seq.M : (long long)a.seq.B * a.seq.T;
    TcBoxes box;
    box.tok_tile = kKeys / a.G;
    box.q_tok = (int)(box.tok_tile < tokens ? box.tok_tile : tokens);
    box.kv_rows = a.cache.S < kKeys ? a.cache.S : kKeys;
    TcMaps maps;
    {
        const cuuint64_t dim[4] = {(cuuint64_t)D, (cuuint64_t)a.G, (cuuint64_t)a.cache.H, (cuuint64_t)tokens};
        const cuuint64_t stride[3] = {row, row * a.G, row * a.Hq};
        const cuuint32_t bx[4] = {64, (cuuint32_t)a.G, 1, (cuuint32_t)box.q_tok};
        if (!make_map(&maps.q, bf16, a.q, 4, dim, stride, bx))
            return cudaErrorInvalidValue;
    }
    const cuuint64_t slab = row * a.cache.S;
    const char *layer = static_cast<const char *>(a.cache.kv) + a.cache.k_slab * slab;
    {
        const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)a.cache.S, 2ull * a.cache.N * a.cache.H};
        const cuuint64_t stride[2] = {row, slab};
        const cuuint32_t bx[3] = {64, (cuuint32_t)box.kv_rows, 1};
        if (!make_map(&maps.kv, bf16, layer, 3, dim, stride, bx))
            return cudaErrorInvalidValue;
    }
    maps.node = maps.kv;
    box.node_rows = 0;
    if (!PROMPT) {
        const int rows = a.seq.staged ? a.seq.T : a.cache.S;
        box.node_rows = a.seq.T < rows ? a.seq.T : rows;
        const cuuint64_t sl = row * rows, n = a.seq.staged ? 2ull * a.seq.B * a.cache.H : 2ull * a.cache.N * a.cache.H;
        const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)rows, n};
        const cuuint64_t stride[2] = {row, sl};
        const cuuint32_t bx[3] = {64, (cuuint32_t)box.node_rows, 1};
        const char *p = a.seq.staged ? static_cast<const char *>(a.staged) + a.st_k * sl : layer;
        if (!make_map(&maps.node, bf16, p, 3, dim, stride, bx))
            return cudaErrorInvalidValue;
    }
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
    return at % 16 == 0 && encode_tiled() != nullptr;
}

cudaError_t launch_attend_tc(const AttendArgs &a, spec_dtype dt, cudaStream_t st)
{
    if (a.cache.D == 64)
        return dt == SPEC_BF16 ? launch_tc_d<__nv_bfloat16, 64>(a, st) : launch_tc_d<__half, 64>(a, st);
    return dt == SPEC_BF16 ? launch_tc_d<__nv_bfloat16, 128>(a, st) : launch_tc_d<__half, 128>(a, st);
}

size_t attend_tc_workspace(int T, int Hq, int H, int D)
{
    const long long rows = (long long)T * (Hq / (H > 0 ? H : 1));
    const size_t part = rows <= kKeys ? part_floats<128>(D) : part_floats<256>(D);
    return align256(kPartHead + 2 * kAttendCtas * part * sizeof(float));
}

}  // namespace spec
