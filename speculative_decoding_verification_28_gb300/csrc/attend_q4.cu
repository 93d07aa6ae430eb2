// attend_q4.cu -- attention of a round over pages of 4-bit keys and values:
// rounds where a key head has few query rows (decoding, short chains).
//
//   S^T = K Q^T,  P^T = 2^(c S^T - m),  O^T += V^T P^T
//
// Keys and values are the first operands of m16n8k16 products, so that codes go
// from shared memory to registers, become fp16 there and meet the tensor cores:
// written back as 16-bit tiles for tcgen05 they would cost six times the shared
// memory traffic that they arrive with.  A product's summed index may run in any
// order as long as both operands have the same, so lane (g, t) takes the
// dimensions of one run of bytes: t's quarter of key row g, g's eighth of value
// rows 2t, 2t + 1, 2t + 8, 2t + 9.  Expanded values, and so S and O, are 128
// times too small (q4_expand.cuh), which the scale and the last division make good.
//
// Queries are fp16 too, bf16 rows times a power of two.  Weights are fp16, 2^11
// times as large as the softmax's, under a maximum that moves only when a tile
// exceeds it by more than 2^4 (tcgen.cuh says why).  The nodes' tile is in the
// staged type on both sides, weights too.
//
// What it takes: decoding over 70000 keys (6 sequences, 64 / 8 heads of 128) 106 us, HBM's floor
// 68.  1190 instructions a tile of 64 keys, half of them to expand, at half of the issue slots.
//
// A CTA: four warps, each with its own running statistics and every fourth of the
// unit's tiles of 64 keys, joined in shared memory at the unit's end; a fifth walks
// over the units and copies pages' codes and scales (cp.async.bulk) through a ring.
// A slot of the ring is always the same warp's: to a warp that had not waited for the
// slot's tile before, that one's parity would look like its own tile's.
#include <type_traits>

#include "paged_units.cuh"
#include "q4_expand.cuh"

namespace spec {

constexpr int kQ4Keys = 64;  // keys of a tile
constexpr int kQ4Warps = 4;  // that compute
constexpr int kQ4Threads = 32 * (kQ4Warps + 1);

// NQ: query tiles of 8 rows of a unit
template <int D, int NQ>
struct Q4Shape {
    static constexpr int kRows = 8 * NQ;
    static constexpr int kCtas = NQ == 1 ? 3 : 2;  // of an SM
    static constexpr int kStages = 2 * kQ4Warps;
    static constexpr int kCodes = kQ4Keys * q4_codes(D), kScales = kQ4Keys * q4_scales(D);
    static constexpr int kTile = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
    static constexpr int kStride = D + 4;                 // floats of a row in the join
};
template <int D, int NQ>
struct Q4Shared {
    using Sh = Q4Shape<D, NQ>;
    unsigned char ring[Sh::kStages][Sh::kTile];
    float o[Sh::kRows][Sh::kStride];
    float m[kQ4Warps][Sh::kRows], l[Sh::kRows];
    uint64_t full[Sh::kStages], empty[Sh::kStages], never;
    PagedRing units;
    uint32_t scan[kQ4Threads / 32 + 1];
    Run run;
    uint32_t asked;  // tiles that were copied in all
    int abort, last;
};

// among the warps that compute
__device__ __forceinline__ void q4_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// ... and whether all of them say so.  They go on to a unit together or not at
// all: after a wait that gave up, one that left alone would be waited for above.
__device__ __forceinline__ bool q4_all(bool yes)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 2, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)yes)
                 : "memory");
    return r != 0;
}
static_assert(32 * kQ4Warps == 128, "q4_sync, q4_all");
static_assert(3 * kAttendCtas <= kGaveUpWord, "one counter per CTA");

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
                 "%2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
                 "%1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 tile of 16-bit values, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// A warp's share of a unit: O^T (rows g * D / 8 + 2 j and the next, columns
// 2 t and the next of each query tile), running maxima and partial sums.
template <int D, int NQ>
struct Q4State {
    float o[NQ][D / 16][4];
    float m[NQ][2], l[NQ][2];
};

// Scores (raw, times c per column) to weights: new maxima, rescaled O, and the
// weights as second operands of O^T += V^T P^T.  NSUB: groups of 16 keys.
template <typename T, int D, int NQ, int NSUB>
__device__ __forceinline__ void q4_softmax(Q4State<D, NQ> &st, float (&s)[NSUB][NQ][4], const float (&c)[NQ][2],
                                           uint32_t (&pb)[NSUB][NQ][2])
{
    constexpr float kShift = TcType<__half>::kShift, kLazy = TcType<__half>::kLazy;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[0][q][e], s[0][q][e + 2]);
#pragma unroll
            for (int i = 1; i < NSUB; ++i)
                x = max3(x, s[i][q][e], s[i][q][e + 2]);
            mx[e] = x;
        }
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xFFFFFFFFu, mx[0], k));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xFFFFFFFFu, mx[1], k));
        }
        mx[0] *= c[q][0];
        mx[1] *= c[q][1];
        if (__any_sync(0xFFFFFFFFu, mx[0] > st.m[q][0] + kLazy || mx[1] > st.m[q][1] + kLazy)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float f = 1.0f;
                if (mx[e] > st.m[q][e] + kLazy) {
                    f = exp2_sfu(st.m[q][e] - mx[e]);  // 0 when nothing was seen before
                    st.m[q][e] = mx[e];
                }
                st.l[q][e] *= f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    st.o[q][j][e] *= f;
                    st.o[q][j][e + 2] *= f;
                }
            }
        }
        float b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            b[e] = kShift - (st.m[q][e] == -INFINITY ? 0.0f : st.m[q][e]);
#pragma unroll
        for (int i = 0; i < NSUB; ++i) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = exp2_sfu(fmaf(s[i][q][e], c[q][e & 1], b[e & 1]));
            st.l[q][0] += p[0] + p[2];
            st.l[q][1] += p[1] + p[3];
            pb[i][q][0] = transposed(TcType<T>::pack(p[0], p[1]));
            pb[i][q][1] = transposed(TcType<T>::pack(p[2], p[3]));
        }
    }
}

// One tile of 4-bit keys and values; `valid` of its keys count.
template <int D, int NQ>
__device__ __forceinline__ void q4_tile(Q4State<D, NQ> &st, unsigned char *tile, int valid,
                                        const uint32_t (&qf)[NQ][D / 16][2], const float (&c)[NQ][2])
{
    using Sh = Q4Shape<D, NQ>;
    constexpr int NSUB = kQ4Keys / 16, KW = D / 32, VW = D / 64;  // words of a lane: of a key row, of a value row
    constexpr int kScales = q4_scales(D);
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    unsigned char *vs = tile + 2 * Sh::kCodes + Sh::kScales;
    if (valid < kQ4Keys) {
        // values behind the last key have no weight, but what lies there may be anything
        for (int row = valid + lane; row < kQ4Keys; row += 32)
#pragma unroll
            for (int i = 0; i < kScales; ++i)
                vs[row * kScales + i] = 0;
        __syncwarp();
    }
    const unsigned char *kc = tile + g * q4_codes(D) + t * KW * 4;
    const unsigned char *ks = tile + 2 * Sh::kCodes + g * kScales + t * kScales / 4;
    float s[NSUB][NQ][4];
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
        uint32_t w[2][KW];
        uint32_t sc[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 16 * i + 8 * r;
            if constexpr (KW == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(kc + row * q4_codes(D));
                w[r][0] = x.x, w[r][1] = x.y, w[r][2] = x.z, w[r][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(kc + row * q4_codes(D));
                w[r][0] = x.x, w[r][1] = x.y;
            }
            sc[r] = (uint32_t)ks[row * kScales] * 0x00800080u;
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[i][q][e] = 0.0f;
        const Scale2 s0(sc[0]), s1(sc[1]);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            uint32_t x0[4], x1[4];
            q4_expand(w[0][k], s0, x0);
            q4_expand(w[1][k], s1, x1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t a[4] = {x0[2 * h], x1[2 * h], x0[2 * h + 1], x1[2 * h + 1]};
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    mma16816<__half>(s[i][q], a, qf[q][2 * k + h][0], qf[q][2 * k + h][1]);
            }
        }
    }
    if (valid < kQ4Keys) {
#pragma unroll
        for (int i = 0; i < NSUB; ++i)
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                if (16 * i + g >= valid)
                    s[i][q][0] = s[i][q][1] = -INFINITY;
                if (16 * i + 8 + g >= valid)
                    s[i][q][2] = s[i][q][3] = -INFINITY;
            }
    }
    uint32_t pb[NSUB][NQ][2];
    q4_softmax<__half, D, NQ, NSUB>(st, s, c, pb);
    const unsigned char *vc = tile + Sh::kCodes + 2 * t * q4_codes(D) + g * VW * 4;
    const unsigned char *vsl = vs + 2 * t * kScales + g * kScales / 8;
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
        uint32_t a[2][8 * VW];  // [pair of keys][dimension]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 16 * i + 8 * r;
            const uint32_t *pa = reinterpret_cast<const uint32_t *>(vc + row * q4_codes(D));
            const uint32_t *pn = reinterpret_cast<const uint32_t *>(vc + (row + 1) * q4_codes(D));
            uint32_t wa[VW], wb[VW];
#pragma unroll
            for (int k = 0; k < VW; ++k) {
                wa[k] = pa[k];
                wb[k] = pn[k];
            }
            const uint32_t sa = vsl[row * kScales], sb = vsl[(row + 1) * kScales];
            const Scale2 s2((sa | sb << 16) << 7);
#pragma unroll
            for (int k = 0; k < VW; ++k) {
                q4_expand(__byte_perm(wa[k], wb[k], 0x5410), s2, a[r] + 8 * k);
                q4_expand(__byte_perm(wa[k], wb[k], 0x7632), s2, a[r] + 8 * k + 4);
            }
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const uint32_t v[4] = {a[0][2 * j], a[0][2 * j + 1], a[1][2 * j], a[1][2 * j + 1]};
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                mma16816<__half>(st.o[q][j], v, pb[i][q][0], pb[i][q][1]);
        }
    }
    if (valid < kQ4Keys)  // the zeros above come before the slot's next copy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Adds what is not finite among the nodes' values (taken out of the products: a
// weight of 0 times it would reach rows that do not see it) to the rows that do.
// Their weights are positive, so that it stays as it is.
template <typename T, int D, int NQ>
__device__ __noinline__ void q4_put_back(const AttendArgs &a, const PagedUnit &u, const T *values, float *o)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int q = 0; q < NQ; ++q)
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * q + 2 * t + e;
            if (r >= u.n_rows)
                continue;
            const uint64_t bits = row_nodes(a, u, r);
            for (int key = 0; key < u.n; ++key)
                if (bits >> key & 1)
                    for (int d = 0; d < D / 8; ++d) {
                        const float f = Storage<T>::at(values + (size_t)key * D, g * (D / 8) + d);
                        if (!(fabsf(f) <= 3.4e38f))
                            o[(q * (D / 16) + d / 2) * 4 + e + 2 * (d & 1)] += f;
                    }
        }
}

// The nodes' tile: 16-bit keys and values from global memory, masks.
template <typename T, int D, int NQ>
__device__ __noinline__ void q4_nodes(const AttendArgs &a, const PagedUnit &u, Q4State<D, NQ> &to)
{
    Q4State<D, NQ> st = to;
    constexpr int NSUB = SPEC_MAX_NODES / 16, KV = D / 32, VV = D / 64;  // 16-byte words of a lane: key row, value row
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, n = u.n;
    const T *keys = reinterpret_cast<const T *>(a.staged) + (a.st_k + (long long)u.b * a.cache.H + u.h) * a.seq.T * D;
    const T *values = reinterpret_cast<const T *>(a.staged) + (a.st_v + (long long)u.b * a.cache.H + u.h) * a.seq.T * D;
    // the nodes' products are in the storage type, and O in its own units
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                st.o[q][j][e] *= 128.0f;
    float s[NSUB][NQ][4], c[NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        c[q][0] = c[q][1] = a.scale_log2;
        uint32_t qf[D / 16][2];
        const int r = 8 * q + g;
        const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.q) +
                                                         row_place(a, u, min(r, u.n_rows - 1)) + t * (D / 4));
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            uint32_t x[4];
            pairs_of(__ldg(p + k), x);
            qf[2 * k][0] = x[0], qf[2 * k][1] = x[1], qf[2 * k + 1][0] = x[2], qf[2 * k + 1][1] = x[3];
        }
        uint64_t bits[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            bits[e] = 8 * q + 2 * t + e < u.n_rows ? row_nodes(a, u, 8 * q + 2 * t + e) : 0;
#pragma unroll
        for (int i = 0; i < NSUB; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[i][q][e] = 0.0f;
            if (16 * i < n) {
                uint32_t x[2][KV][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 *kp =
                        reinterpret_cast<const uint4 *>(keys + (size_t)min(16 * i + 8 * h + g, n - 1) * D + t * (D / 4));
#pragma unroll
                    for (int k = 0; k < KV; ++k)
                        pairs_of(__ldg(kp + k), x[h][k]);
                }
#pragma unroll
                for (int k = 0; k < KV; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t f[4] = {x[0][k][2 * h], x[1][k][2 * h], x[0][k][2 * h + 1], x[1][k][2 * h + 1]};
                        mma16816<T>(s[i][q], f, qf[2 * k + h][0], qf[2 * k + h][1]);
                    }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(bits[e & 1] >> (16 * i + 8 * (e >> 1) + g) & 1))
                    s[i][q][e] = -INFINITY;
        }
    }
    uint32_t pb[NSUB][NQ][2];
    q4_softmax<T, D, NQ, NSUB>(st, s, c, pb);
    bool odd = false;
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
        if (16 * i >= n)
            break;
        uint32_t v[2][VV][2][4];  // [pair of keys][16-byte word of a row][key][pairs of dimensions]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 16 * i + 8 * h + 2 * t + e;
                const uint4 *vp = reinterpret_cast<const uint4 *>(values + (size_t)min(row, n - 1) * D + g * (D / 8));
#pragma unroll
                for (int k = 0; k < VV; ++k) {
                    uint4 x = __ldg(vp + k);
                    if (row >= n)
                        x = make_uint4(0, 0, 0, 0);
                    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        uint32_t z = y[d];
                        if ((z & TcType<T>::kExp) == TcType<T>::kExp) {
                            z &= 0xFFFF0000u;
                            odd = true;
                        }
                        if ((z >> 16 & TcType<T>::kExp) == TcType<T>::kExp) {
                            z &= 0x0000FFFFu;
                            odd = true;
                        }
                        v[h][k][e][d] = z;
                    }
                }
            }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const int k = j / 4, d = j % 4;
            const uint32_t f[4] = {
                __byte_perm(v[0][k][0][d], v[0][k][1][d], 0x5410), __byte_perm(v[0][k][0][d], v[0][k][1][d], 0x7632),
                __byte_perm(v[1][k][0][d], v[1][k][1][d], 0x5410), __byte_perm(v[1][k][0][d], v[1][k][1][d], 0x7632)};
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                mma16816<T>(st.o[q][j], f, pb[i][q][0], pb[i][q][1]);
        }
    }
    if (__any_sync(0xFFFFFFFFu, odd)) {
        Q4State<D, NQ> x = st;
        q4_put_back<T, D, NQ>(a, u, values, &x.o[0][0][0]);
        st = x;
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                st.o[q][j][e] *= 0.0078125f;
    to = st;
}

// A unit's queries as second operands, fp16, and the factor that takes a raw
// score to base 2, per column.
template <typename T, int D, int NQ>
__device__ __forceinline__ void q4_queries(const AttendArgs &a, const PagedUnit &u, uint32_t (&qf)[NQ][D / 16][2],
                                           float (&c)[NQ][2])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int r = 8 * q + g;
        const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.q) +
                                                         row_place(a, u, min(r, u.n_rows - 1)) + t * (D / 4));
        uint32_t w[D / 32][4];
        int e = 0;
        if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                pairs_of(__ldg(p + k), w[k]);
        } else {
            float x[D / 32][8], top = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                Storage<T>::unpack(__ldg(p + k), x[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = fmaxf(top, fabsf(x[k][i]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const bool small = top < 1.0f / kSmallRow;
            if (small) {
                top *= kSmallRow;
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[k][i] *= kSmallRow;
            }
            e = q4_row_exponent(top);
            const float f = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[k][i] = TcType<__half>::pack(x[k][i] * f, x[k][i + 4] * f);
            e += small ? 64 : 0;
        }
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            qf[q][2 * k][0] = w[k][0], qf[q][2 * k][1] = w[k][1];
            qf[q][2 * k + 1][0] = w[k][2], qf[q][2 * k + 1][1] = w[k][3];
        }
        // a column's factor comes from a lane that has its row; never 0, which would make
        // hidden scores NaN (raw ones are below 2^25, so that nothing else sees the limit)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c[q][i] = fmaxf(a.scale_log2 * exp2f((float)(7 - __shfl_sync(0xFFFFFFFFu, e, (2 * t + i) * 4))),
                            1.17549435e-38f);
    }
}

template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kQ4Threads, Q4Shape<D, NQ>::kCtas) attend_q4_kernel(const __grid_constant__ AttendQ4Args x)
{
    using Sh = Q4Shape<D, NQ>;
    constexpr int ST = Sh::kStages;
    extern __shared__ __align__(128) unsigned char base[];
    Q4Shared<D, NQ> &s = *reinterpret_cast<Q4Shared<D, NQ> *>(base);
    const AttendArgs &a = x.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // A unit's start and end cost about eight tiles.  Counted as none / 4 / 8 / 16, us (8 key heads, 500 .. 4000
    // keys unless said): 128 sequences of 4 rows 117 / 107 / 98 / 97; 64 of 12 rows 125 / 106 / 96 / 94, of 16
    // with heads of 64 77 / 65 / 59 / 56; 32 of 1 row, 2000 keys 31 / 29 / 27 / 29; long ones 112 / 110 / 110 / 107.
    // Only 64 of 4 rows with heads of 64 would rather have none, 53 / 55 / 59 / 64.
    const UnitShape<8> sh{kQ4Keys, Sh::kRows, a.G};
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        units_init(s.units, kQ4Warps);
        mbar_init(&s.never, 1);
        fence_mbar_init();
        s.abort = 0;
        s.asked = 0;
        s.run.begin = s.run.end = 0;
    }
    __syncthreads();  // run.begin / end above come before find_run's
    find_run<kQ4Threads, false>(a, sh, s.scan, &s.run);
    __syncthreads();
    const long long limit = a.wait_clocks;

    if (warp == kQ4Warps) {
        // ------------------------------------------------------------ loads
        UnitWalk<UnitShape<8>> walk(a, sh, s.run);
        AttendUnit w{};
        TileCopies<D, kQ4Keys> copies(x);
        uint32_t it = 0, n = 0;
        bool ok = true;
        while (ok && walk.next(w)) {
            ok = units_put(s.units, n++, &w, &s.abort, limit);
            prefetch_unit<T, D>(a, w);
            copies.begin(w);
            const int end = min(w.tile_end, w.n_tiles - 1);
            for (int tile = w.tile; ok && tile < end; ++tile, ++it) {
                const int sg = it % ST, page = copies.template page_of<true>(tile);
                ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.empty[sg], ((it / ST) & 1) ^ 1, &s.abort, limit));
                if (!ok)
                    break;
                copies.issue(tile, page, s.ring[sg], &s.full[sg]);
            }
        }
        if (ok)
            units_put(s.units, n, nullptr, &s.abort, limit);
        if (lane == 0)
            s.asked = it;
        paged_flags(x, sh, s.run);
    } else {
        // ---------------------------------------------------------- compute
        const int g = lane >> 2, t = lane & 3;
        uint32_t it = 0;  // tiles through the ring
        bool ok = !a.starve || __all_sync(0xFFFFFFFFu, wait_phase(&s.never, 0, &s.abort, limit));
        for (uint32_t n = 0; q4_all(units_wait(s.units, n, &s.abort, limit)); ++n) {
            const PagedUnit &u = *units_at(s.units, n);  // read as it is wanted: registers are short
            Q4State<D, NQ> st;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                st.m[q][0] = st.m[q][1] = -INFINITY;
                st.l[q][0] = st.l[q][1] = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        st.o[q][j][e] = 0.0f;
            }
            const int tiles = max(0, min(u.tile_end, u.n_tiles - 1) - u.tile);  // of the prefix
            const int j0 = (warp - (int)it) & (kQ4Warps - 1);
            if (ok && j0 < tiles) {
                uint32_t qf[NQ][D / 16][2];
                float c[NQ][2];
                q4_queries<T, D, NQ>(a, u, qf, c);
                for (int j = j0; ok && j < tiles; j += kQ4Warps) {
                    const uint32_t i = it + j, sg = i % ST;
                    ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.full[sg], (i / ST) & 1, &s.abort, limit));
                    if (!ok)
                        break;
                    q4_tile<D, NQ>(st, s.ring[sg], min(kQ4Keys, u.prefix - (u.tile + j) * kQ4Keys), qf, c);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&s.empty[sg]);
                }
            }
            it += tiles;
            // the next warp in turn has the nodes
            if (ok && u.tile_end == u.n_tiles && (it & (kQ4Warps - 1)) == warp) {
                Q4State<D, NQ> y = st;  // the call keeps only this copy in memory
                q4_nodes<T, D, NQ>(a, u, y);
                st = y;
            }
            // The warps' parts, under a common maximum, added up by the first, one
            // after another: a buffer for each would cost the ring its second slots.
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1)
                        st.l[q][e] += __shfl_xor_sync(0xFFFFFFFFu, st.l[q][e], k);
                    if (g == 0)
                        s.m[warp][8 * q + 2 * t + e] = st.m[q][e];
                }
            q4_sync();
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * q + 2 * t + e;
                    float m = s.m[0][r];
#pragma unroll
                    for (int w = 1; w < kQ4Warps; ++w)
                        m = fmaxf(m, s.m[w][r]);
                    const float f = exp2f(st.m[q][e] - (m == -INFINITY ? 0.0f : m));
                    st.m[q][e] = m;
                    st.l[q][e] *= f;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        st.o[q][j][e] *= f * kQ4Units;
                        st.o[q][j][e + 2] *= f * kQ4Units;
                    }
                }
#pragma unroll 1
            for (int w = 1; w < kQ4Warps; ++w) {
                if (warp == w) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float *row = s.o[8 * q + 2 * t + e] + g * (D / 8);
#pragma unroll
                            for (int j = 0; j < D / 16; j += 2)
                                *reinterpret_cast<float4 *>(row + 2 * j) = make_float4(
                                    st.o[q][j][e], st.o[q][j][e + 2], st.o[q][j + 1][e], st.o[q][j + 1][e + 2]);
                            if (g == 0)
                                s.l[8 * q + 2 * t + e] = st.l[q][e];
                        }
                }
                q4_sync();
                if (warp == 0) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float *row = s.o[8 * q + 2 * t + e] + g * (D / 8);
#pragma unroll
                            for (int j = 0; j < D / 16; j += 2) {
                                const float4 z = *reinterpret_cast<const float4 *>(row + 2 * j);
                                st.o[q][j][e] += z.x;
                                st.o[q][j][e + 2] += z.y;
                                st.o[q][j + 1][e] += z.z;
                                st.o[q][j + 1][e + 2] += z.w;
                            }
                            st.l[q][e] += s.l[8 * q + 2 * t + e];
                        }
                }
                q4_sync();
            }
            const bool whole = u.n_parts == 1;
            if (warp == 0) {
                float *slot = whole ? nullptr : part_slot<Sh::kRows>(a, blockIdx.x, u.part);
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 8 * q + 2 * t + e;
                        if (r >= u.n_rows)
                            continue;
                        const float l = st.l[q][e], to = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                        T *dst = reinterpret_cast<T *>(a.out) + row_place(a, u, r) + g * (D / 8);
#pragma unroll
                        for (int j = 0; j < D / 16; j += 4) {
                            const float y[8] = {st.o[q][j][e],     st.o[q][j][e + 2],     st.o[q][j + 1][e], st.o[q][j + 1][e + 2],
                                                st.o[q][j + 2][e], st.o[q][j + 2][e + 2], st.o[q][j + 3][e], st.o[q][j + 3][e + 2]};
                            if (whole) {
                                uint4 v;
                                v.x = TcType<T>::pack(y[0] * to, y[1] * to);
                                v.y = TcType<T>::pack(y[2] * to, y[3] * to);
                                v.z = TcType<T>::pack(y[4] * to, y[5] * to);
                                v.w = TcType<T>::pack(y[6] * to, y[7] * to);
                                *reinterpret_cast<uint4 *>(dst + 2 * j) = v;
                            } else {
                                const int d = (g * (D / 8) + 2 * j) / 4;
                                __stcg(reinterpret_cast<float4 *>(slot + part_quad<Sh::kRows>(d, r)),
                                       make_float4(y[0], y[1], y[2], y[3]));
                                __stcg(reinterpret_cast<float4 *>(slot + part_quad<Sh::kRows>(d + 1, r)),
                                       make_float4(y[4], y[5], y[6], y[7]));
                            }
                        }
                        if (!whole && g == 0) {
                            __stcg(slot + (size_t)Sh::kRows * D + r, st.m[q][e]);
                            __stcg(slot + (size_t)Sh::kRows * D + Sh::kRows + r, l);
                        }
                    }
            }
            if (!whole) {
                if (warp == 0) {
                    __threadfence();
                    __syncwarp();
                    if (lane == 0) {
                        s.last = 0;
                        if (!*reinterpret_cast<volatile int *>(&s.abort)) {
                            int *cnt = part_counter(a, u.first_cta);
                            s.last = atomicAdd(cnt, 1) == u.n_parts - 1;
                            if (s.last)
                                *cnt = 0;
                        }
                    }
                }
                q4_sync();
                if (s.last) {
                    __threadfence();
                    join_parts<T, Sh::kRows>(a, join_unit(a, u), tid, 32 * kQ4Warps, [] {
                        __threadfence();
                        q4_sync();
                        return true;
                    });
                }
                q4_sync();  // `last` has been read
            }
            units_done(s.units, n);
        }
    }
    __syncthreads();
    if (s.abort && warp == kQ4Warps) {
        if (lane == 0)
            await_copies<ST>(s.full, s.asked);
        __syncwarp();
        give_up(a);
    }
}

namespace {

template <typename T, int D, int NQ>
cudaError_t launch_q4(const AttendQ4Args &a, cudaStream_t st)
{
    constexpr int smem = (int)sizeof(Q4Shared<D, NQ>);
    static_assert(smem * Q4Shape<D, NQ>::kCtas <= 232448 - 1024 * Q4Shape<D, NQ>::kCtas, "CTAs of an SM");
    const cudaError_t e =
        cudaFuncSetAttribute(attend_q4_kernel<T, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    attend_q4_kernel<T, D, NQ><<<kAttendCtas * Q4Shape<D, NQ>::kCtas, kQ4Threads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_q4_d(const AttendQ4Args &a, cudaStream_t st)
{
    // Query rows of a key head decide.  Measured on both sides (500 .. 4000 keys, 8 key heads of 128, us):
    //   1 .. 8 rows   one query tile here 97 (128 sequences of 4 rows), two 153, tcgen05 180; heads of 64 59, 72, 105
    //   9 .. 16       two tiles 91 (64 of 12), one (two units) 96, tcgen05 99; heads of 64 (16 rows) 58, 67, 84
    //   17 and more   tcgen05 100 (64 of 20), units of 16 rows here 168, of 8 136
    // Batches of 8 and 16 over 50 .. 400 keys and 2 key heads take 18 .. 21 in any form.  The rule is made for
    // batches: 4 sequences over 20000 .. 40000 keys, 2 key heads of 64, would rather have tcgen05 from 8 rows on
    // (8 rows 45, 39, 33; 16 rows 40, 37, 33; 20 rows 37 in all).
    const int rows = a.a.seq.T * a.a.G;
    if (rows > 16)
        return launch_attend_q4_tc(a, std::is_same<T, __half>::value ? SPEC_F16 : SPEC_BF16, st);
    return rows <= 8 ? launch_q4<T, D, 1>(a, st) : launch_q4<T, D, 2>(a, st);
}

}  // namespace

cudaError_t launch_attend_q4(const AttendQ4Args &a, spec_dtype dt, cudaStream_t st)
{
    if (a.pool.D == 64)
        return dt == SPEC_BF16 ? launch_q4_d<__nv_bfloat16, 64>(a, st) : launch_q4_d<__half, 64>(a, st);
    return dt == SPEC_BF16 ? launch_q4_d<__nv_bfloat16, 128>(a, st) : launch_q4_d<__half, 128>(a, st);
}

size_t attend_q4_workspace(int D)
{
    const size_t one = 2 * 3 * kAttendCtas * part_floats<8>(D), many = 2 * 2 * kAttendCtas * part_floats<16>(D);
    const size_t few = align256(kPartHead + (one > many ? one : many) * sizeof(float)), tc = attend_q4_tc_workspace(D);
    return few > tc ? few : tc;
}

}  // namespace spec
