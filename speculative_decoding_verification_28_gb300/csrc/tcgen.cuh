// tcgen.cuh -- the fifth-generation tensor core's instructions (tcgen05, TMEM,
// TMA tensor loads) as this library's attention kernels use them on sm_103a,
// and the parts those kernels share: bounded waits, the guard of V tiles, the
// tensor maps.
#pragma once

#include <cuda.h>

#include "attend_common.cuh"
#include "bulk_copy.cuh"
#include "packed.cuh"
#include "verify_common.cuh"

namespace spec {

constexpr int kKeys = 128;  // keys of a tile
constexpr int kTcWaitLimit = 2000;  // probes of up to ~1 ms, after a wait that gave up
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
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : SPEC_OUT4(r, 0), SPEC_OUT4(r, 4), SPEC_OUT4(r, 8), SPEC_OUT4(r, 12)
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

// kShift: weights are 2^kShift times as large as the softmax's; kLazy: base-2
// headroom of the running maximum.  An fp16 weight of less than 2^-14 has steps
// of 2^-24: unshifted, weights under 2^-25 of a row's largest would all be 0, and
// thousands of them may be most of its result.  At 2^11 they keep their 11 bits
// down to 2^-25 and vanish under 2^-36, and 2^(11 + 4) is within fp16's range.
// bf16 has fp32's range.
template <typename T>
struct TcType;
template <>
struct TcType<__nv_bfloat16> {
    static constexpr uint32_t kFmt = 1;
    static constexpr float kShift = 0.0f, kLazy = 8.0f;
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
    static constexpr float kShift = 11.0f, kLazy = 4.0f;
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

// 32 columns of a row times f, rounded, to 16-byte aligned dst.  A thread
// writes a row of its own, so whole 32-byte sectors at a time where it may.
template <typename T>
__device__ __forceinline__ void store_row32(T *dst, const uint32_t *o, float f)
{
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
        w[e] = TcType<T>::pack(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
    if (reinterpret_cast<uintptr_t>(dst) % 32 == 0) {
#pragma unroll
        for (int e = 0; e < 16; e += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 2 * e), SPEC_IN4(w, e),
                         SPEC_IN4(w, e + 4)
                         : "memory");
    } else {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4 *>(dst + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
    }
}

// Columns 32 k .. of a tile that a row sees, as a word: the first `lim`, or
// for nodes those with their bit set.
__device__ __forceinline__ uint32_t seen32(bool nodes, uint64_t bits, int lim, int k)
{
    if (nodes)
        return (uint32_t)(bits >> (32 * k));
    return lim >= 32 * k + 32 ? ~0u : lim <= 32 * k ? 0u : (1u << (lim - 32 * k)) - 1;
}
// scores that are not seen: -inf
__device__ __forceinline__ void hide32(uint32_t *v, uint32_t seen)
{
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!(seen >> e & 1))
            v[e] = 0xFF800000u;
}

// instruction descriptor: fp32 accumulators, both operands T, M = 128
template <typename T>
__device__ __forceinline__ uint32_t tc_idesc(int n, bool b_rows_summed)
{
    return (1u << 4) | (TcType<T>::kFmt << 7) | (TcType<T>::kFmt << 10) | ((b_rows_summed ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

struct TcMaps {
    CUtensorMap q, kv, node;
};
// rows the maps' boxes bring
struct TcBoxes {
    int q_tok, tok_tile, kv_rows, node_rows;
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

// The guard's work on a V tile (panels of kKeys rows of 128 bytes), by a whole
// warp: rows that the product reads past the last key are zeroed; in a tile
// with places that some rows do not see, values that are not finite are taken
// out (a weight of 0 times them would reach those rows) and their keys noted
// in odd[4 g ..], g the unit's masked tiles so far, and odd[12].
template <typename T, int PANELS>
__device__ __forceinline__ void guard_tile(unsigned char *v, const Tile &tl, uint32_t *odd, int &g)
{
    constexpr int kPanel = kKeys * 128;
    const int lane = threadIdx.x & 31;
    for (int r = tl.valid + (lane >> 3); r < ((tl.valid + 15) & ~15); r += 4)
#pragma unroll
        for (int p = 0; p < PANELS; ++p)
            *reinterpret_cast<uint4 *>(v + p * kPanel + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
    if (tl.masked) {
        uint32_t m = 0;
        for (int r = lane >> 3; r < tl.valid; r += 4)
#pragma unroll
            for (int p = 0; p < PANELS; ++p) {
                const uint4 x = *reinterpret_cast<const uint4 *>(v + p * kPanel + r * 128 + (lane & 7) * 16);
                m = TcType<T>::max_abs(TcType<T>::max_abs(m, x.x), x.y);
                m = TcType<T>::max_abs(TcType<T>::max_abs(m, x.z), x.w);
            }
        if (__any_sync(0xFFFFFFFFu, TcType<T>::odd(m))) {  // rare
            odd[12] = 1;
            for (int r = lane >> 3; r < tl.valid; r += 4)
                for (int p = 0; p < PANELS; ++p) {
                    uint32_t *w = reinterpret_cast<uint32_t *>(v + p * kPanel + r * 128 + (lane & 7) * 16);
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
        ++g;
    }
    __threadfence_block();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// V row of key `key` of a tile, in global memory
template <typename T>
__device__ __forceinline__ const T *value_row(const AttendArgs &a, const AttendUnit &u, const Tile &tl, int tile, int key)
{
    const int D = a.cache.D;
    if (tl.nodes && a.seq.staged)
        return reinterpret_cast<const T *>(a.staged) +
               ((a.st_v + (long long)u.b * a.cache.H + u.h) * a.seq.T + key) * D;
    return reinterpret_cast<const T *>(a.cache.kv) +
           ((a.cache.v_slab + (long long)u.seq.row * a.cache.H + u.h) * a.cache.S + u.seq.slot0 +
            (tl.nodes ? u.seq.prefix : tile * kKeys) + key) *
               D;
}

// Adds the values that the guard took out of V to columns col .. col + 31 of
// the row of query token `tok`, where it sees their keys.  Their weights are
// positive, so that what is not finite stays as it is.
template <typename T, bool PROMPT>
__device__ __noinline__ void put_back32(const AttendArgs &a, const AttendUnit &u, const uint32_t *odd, int tok, int col,
                                        uint32_t *o)
{
    int g = 0;
    for (int tile = u.tile; tile < u.tile_end; ++tile) {
        const Tile tl = tile_of<PROMPT>(u, tile);
        if (!tl.masked)
            continue;
        for (int key = 0; key < tl.valid; ++key) {
            if (!(odd[g * 4 + (key >> 5)] >> (key & 31) & 1))
                continue;
            bool sees;
            if (tl.nodes)
                sees = (a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1) >> key & 1;
            else
                sees = tile * kKeys + key <= u.seq.prefix + tok;
            if (!sees)
                continue;
            const T *v = value_row<T>(a, u, tl, tile, key) + col;
            for (int e = 0; e < 32; ++e) {
                const float f = Storage<T>::at(v, e);
                if (!(fabsf(f) <= 3.4e38f))
                    o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
            }
        }
        ++g;
    }
}

// Walks the units of a CTA: a prompt's one, or a round's run.
template <bool PROMPT>
struct Units {
    UnitWalk<> walk;
    AttendUnit one;
    bool fresh;
    // some: whether the prompt has one for this CTA
    __device__ Units(const AttendArgs &a, const Shape &sh, const Run &r, const AttendUnit &u, bool some)
        : walk(a, sh, r), one(u), fresh(some)
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

// Bounded wait of one thread for a phase; after one that gave up (`abort`
// set) every other wait of the CTA returns too.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, int *abort, long long limit)
{
    if (mbar_poll(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_poll(bar, parity)) {
        if (*reinterpret_cast<volatile int *>(abort))
            return false;
        if (clock64() - t0 > limit) {
            *reinterpret_cast<volatile int *>(abort) = 1;
            return false;
        }
    }
    return true;
}

// What a CTA whose waits gave up does before it frees TMEM and leaves: its own
// copies into shared memory and its own products have to land first (each with
// a bounded wait), or they would write to memory that is another CTA's by then.
// The last `n` copies into a ring of RING barriers; one thread.
template <int RING>
__device__ __forceinline__ void await_copies(uint64_t *full, uint32_t n)
{
    for (uint32_t i = n > RING ? n - RING : 0; i < n; ++i)
        for (int k = 0; k < kTcWaitLimit && !mbar_try_wait(&full[i % RING], (i / RING) & 1); ++k)
            ;
}
// All products; by the warp that issued them.
__device__ __forceinline__ void await_products(uint64_t *bar)
{
    if (elect_one())
        tc_commit(bar);
    for (int k = 0; k < kTcWaitLimit && !mbar_try_wait(bar, 0); ++k)
        ;
    __syncwarp();
}

// K and V tile of a unit: one box of the cache's map or the nodes' map per
// panel of 64 columns
struct KvBox {
    const CUtensorMap *m;
    int y, z, zv;  // row, K slab, slabs from K to V
    uint32_t bytes;
};
template <int PANELS>
__device__ __forceinline__ KvBox kv_box(const AttendArgs &a, const TcMaps &maps, const TcBoxes &box, const AttendUnit &u,
                                        int tile, bool nodes)
{
    const bool st = nodes && a.seq.staged;
    KvBox k;
    k.m = nodes ? &maps.node : &maps.kv;
    k.y = st ? 0 : u.seq.slot0 + (nodes ? u.seq.prefix : tile * kKeys);
    k.z = st ? u.b * a.cache.H + u.h : u.seq.row * a.cache.H + u.h;
    k.zv = st ? a.seq.B * a.cache.H : a.cache.N * a.cache.H;
    k.bytes = PANELS * 128 * (nodes ? box.node_rows : box.kv_rows);
    return k;
}

// host: the three maps of a call; false if the driver refuses one
bool tc_make_maps(const AttendArgs &a, bool bf16, int tile_rows, TcMaps *maps, TcBoxes *box);
bool tc_available();

}  // namespace spec
