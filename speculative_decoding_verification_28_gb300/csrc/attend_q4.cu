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
// A CTA: four warps, each with its own running statistics and its share of the
// unit's tiles of 64 keys, joined in shared memory at the unit's end; a fifth
// copies pages' codes and scales (cp.async.bulk) through a ring.
#include <type_traits>

#include "attend_common.cuh"
#include "bulk_copy.cuh"
#include "paged.h"
#include "q4_expand.cuh"
#include "tcgen.cuh"

namespace spec {

constexpr int kQ4Keys = 64;  // keys of a tile
constexpr int kQ4Warps = 4;  // that compute
constexpr int kQ4Threads = 32 * (kQ4Warps + 1);

// NQ: query tiles of 8 rows of a unit
template <int D, int NQ>
struct Q4Shape {
    static constexpr int kRows = 8 * NQ;
    static constexpr int kCtas = NQ == 1 ? 3 : 2;  // of an SM
    static constexpr int kStages = D == 64 ? 8 : NQ == 2 ? 8 : 6;
    static constexpr int kCodes = kQ4Keys * q4_codes(D), kScales = kQ4Keys * q4_scales(D);
    static constexpr int kTile = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
    static constexpr int kStride = D + 4;                 // floats of a row in the join
};
template <int D, int NQ>
struct Q4Shared {
    using Sh = Q4Shape<D, NQ>;
    unsigned char ring[Sh::kStages][Sh::kTile];
    float o[kQ4Warps][Sh::kRows][Sh::kStride];
    float m[kQ4Warps][Sh::kRows], l[kQ4Warps][Sh::kRows];
    uint64_t full[Sh::kStages], empty[Sh::kStages], never;
    uint32_t scan[kQ4Threads / 32 + 1];
    Run run;
    uint32_t asked;  // tiles that were copied in all
    int abort, last;
};

// among the warps that compute
__device__ __forceinline__ void q4_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
static_assert(32 * kQ4Warps == 128, "q4_sync");
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
__device__ __forceinline__ void q4_tile(Q4State<D, NQ> &st, const unsigned char *tile, int valid,
                                        const uint32_t (&qf)[NQ][D / 16][2], const float (&c)[NQ][2])
{
    using Sh = Q4Shape<D, NQ>;
    constexpr int NSUB = kQ4Keys / 16, KW = D / 32, VW = D / 64;  // words of a lane: of a key row, of a value row
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const unsigned char *kc = tile, *vc = tile + Sh::kCodes, *ks = vc + Sh::kCodes, *vs = ks + Sh::kScales;
    float s[NSUB][NQ][4];
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[i][q][e] = 16 * i < valid ? 0.0f : -INFINITY;
        if (16 * i >= valid)
            continue;
        uint32_t w[2][KW];
        uint32_t sc[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 16 * i + 8 * r + g;
            const uint32_t *p = reinterpret_cast<const uint32_t *>(kc + row * q4_codes(D)) + t * KW;
            if constexpr (KW == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p);
                w[r][0] = x.x, w[r][1] = x.y, w[r][2] = x.z, w[r][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[r][0] = x.x, w[r][1] = x.y;
            }
            sc[r] = (uint32_t)ks[row * q4_scales(D) + t * q4_scales(D) / 4] * 0x00800080u;
        }
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
        if (valid < 16 * i + 16) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                if (16 * i + g >= valid)
                    s[i][q][0] = s[i][q][1] = -INFINITY;
                if (16 * i + 8 + g >= valid)
                    s[i][q][2] = s[i][q][3] = -INFINITY;
            }
        }
    }
    uint32_t pb[NSUB][NQ][2];
    q4_softmax<__half, D, NQ, NSUB>(st, s, c, pb);
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
        if (16 * i >= valid)
            break;
        uint32_t a[2][8 * VW][1];  // [pair of keys][dimension]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 16 * i + 8 * r + 2 * t;
            uint32_t wa[VW], wb[VW];
            const uint32_t *pa = reinterpret_cast<const uint32_t *>(vc + row * q4_codes(D)) + g * VW;
            const uint32_t *pn = reinterpret_cast<const uint32_t *>(vc + (row + 1) * q4_codes(D)) + g * VW;
#pragma unroll
            for (int k = 0; k < VW; ++k) {
                wa[k] = pa[k];
                wb[k] = pn[k];
            }
            uint32_t sa = vs[row * q4_scales(D) + g * q4_scales(D) / 8],
                     sb = vs[(row + 1) * q4_scales(D) + g * q4_scales(D) / 8];
            // keys behind the last have no weight, but what lies there may be anything
            sa = row < valid ? sa : 0;
            sb = row + 1 < valid ? sb : 0;
            const Scale2 s2(sa << 7 | sb << 23);
#pragma unroll
            for (int k = 0; k < VW; ++k) {
                uint32_t x[4];
                q4_expand(__byte_perm(wa[k], wb[k], 0x5410), s2, x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    a[r][8 * k + e][0] = x[e];
                q4_expand(__byte_perm(wa[k], wb[k], 0x7632), s2, x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    a[r][8 * k + 4 + e][0] = x[e];
            }
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const uint32_t v[4] = {a[0][2 * j][0], a[0][2 * j + 1][0], a[1][2 * j][0], a[1][2 * j + 1][0]};
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                mma16816<__half>(st.o[q][j], v, pb[i][q][0], pb[i][q][1]);
        }
    }
}

// Adds what is not finite among the nodes' values (taken out of the products: a
// weight of 0 times it would reach rows that do not see it) to the rows that do.
// Their weights are positive, so that it stays as it is.
template <typename T, int D, int NQ>
__device__ __noinline__ void q4_put_back(const AttendArgs &a, const AttendUnit &u, const T *values, float *o)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int q = 0; q < NQ; ++q)
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * q + 2 * t + e;
            if (r >= u.n_rows)
                continue;
            const int tok = (u.row0 + r) / a.G;
            const uint64_t bits = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
            for (int key = 0; key < u.seq.n; ++key)
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
__device__ __noinline__ void q4_nodes(const AttendArgs &a, const AttendUnit &u, Q4State<D, NQ> &to)
{
    Q4State<D, NQ> st = to;
    constexpr int NSUB = SPEC_MAX_NODES / 16, KV = D / 32, VV = D / 64;  // 16-byte words of a lane: key row, value row
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, n = u.seq.n;
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
        for (int e = 0; e < 2; ++e) {
            const int tok = (u.row0 + 8 * q + 2 * t + e) / a.G;
            bits[e] = 8 * q + 2 * t + e >= u.n_rows ? 0
                      : a.mask                      ? a.mask[(size_t)u.b * a.seq.T + tok]
                                                    : (2ull << tok) - 1;
            if (n < 64)
                bits[e] &= (1ull << n) - 1;
        }
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
__device__ __forceinline__ void q4_queries(const AttendArgs &a, const AttendUnit &u, uint32_t (&qf)[NQ][D / 16][2],
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
            e = q4_row_exponent(top);
            const float f = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[k][i] = TcType<__half>::pack(x[k][i] * f, x[k][i + 4] * f);
        }
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            qf[q][2 * k][0] = w[k][0], qf[q][2 * k][1] = w[k][1];
            qf[q][2 * k + 1][0] = w[k][2], qf[q][2 * k + 1][1] = w[k][3];
        }
        // a column's factor comes from a lane that has its row
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c[q][i] = a.scale_log2 * exp2f((float)(7 - __shfl_sync(0xFFFFFFFFu, e, (2 * t + i) * 4)));
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
    const Shape sh{kQ4Keys, Sh::kRows, a.G};
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], kQ4Warps);
        }
        mbar_init(&s.never, 1);
        fence_mbar_init();
        s.abort = 0;
        s.run.begin = s.run.end = 0;
    }
    __syncthreads();  // run.begin / end above come before find_run's
    find_run<kQ4Threads, false>(a, sh, s.scan, &s.run);
    __syncthreads();
    const long long limit = a.wait_clocks;
    UnitWalk units(a, sh, s.run);
    AttendUnit u{};
    uint32_t it = 0;  // tiles through the ring

    if (warp == kQ4Warps) {
        // ------------------------------------------------------------ loads
        const int log2 = x.pool.page_log2, piece = min(kQ4Keys, 1 << log2), per = kQ4Keys / piece;
        const int which = lane & 3, mine = lane >> 2;  // K codes, V codes, K scales, V scales of one piece of a tile
        const int width = which < 2 ? q4_codes(D) : q4_scales(D);
        const int at_tile = (which & 1 ? (which < 2 ? Sh::kCodes : Sh::kScales) : 0) + (which < 2 ? 0 : 2 * Sh::kCodes);
        const long long first = which & 1 ? x.v_block : x.k_block;
        bool ok = true;
        while (ok && units.next(u)) {
            const int32_t *row = x.pool.table + (size_t)u.seq.row * x.pool.MP;
            const int end = min(u.tile_end, u.n_tiles - 1);
            int have = -1, held = 0;  // table entry of piece `have` + lane of the sequence
            for (int tile = u.tile; ok && tile < end; ++tile, ++it) {
                const int sg = it % ST, valid = min(kQ4Keys, u.seq.prefix - tile * kQ4Keys);
                const int p0 = tile * per;
                if (have < 0 || p0 + per > have + 32) {
                    have = p0;
                    const long long tok = (long long)(p0 + lane) * piece;
                    held = tok < u.seq.prefix ? __ldg(row + (tok >> log2)) : 0;
                    held = held >= 0 && held < x.pool.P ? held : 0;  // flagged below
                }
                const int page = __shfl_sync(0xFFFFFFFFu, held, p0 - have + (mine < per ? mine : 0));
                ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.empty[sg], ((it / ST) & 1) ^ 1, &s.abort, limit));
                if (!ok)
                    break;
                const int pieces = (valid + piece - 1) / piece;
                if (lane == 0)
                    mbar_arrive_expect_tx(&s.full[sg], (uint32_t)(pieces * piece * 2 * (q4_codes(D) + q4_scales(D))));
                __syncwarp();
                if (mine < pieces) {
                    const unsigned char *blk = x.pool.pool + (first + (long long)page * x.pool.H + u.h) * x.pool.block;
                    const int in_page = (tile * kQ4Keys) & ((1 << log2) - 1);  // of a piece as long as the tile
                    const long long off = which < 2 ? 0 : (long long)q4_codes(D) << log2;
                    bulk_g2s(s.ring[sg] + at_tile + mine * piece * width, blk + off + (long long)in_page * width,
                             (uint32_t)(piece * width), &s.full[sg]);
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
    } else {
        // ---------------------------------------------------------- compute
        bool ok = true;
        const int g = lane >> 2, t = lane & 3;
        while (units.next(u)) {
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
            if (a.starve)
                ok = __all_sync(0xFFFFFFFFu, ok && wait_phase(&s.never, 0, &s.abort, limit));
            if (tiles > 0) {
                uint32_t qf[NQ][D / 16][2];
                float c[NQ][2];
                q4_queries<T, D, NQ>(a, u, qf, c);
                // Every warp waits for every tile and releases it, though it computes
                // only those whose turn is its own: copies may land out of order, and
                // to a warp that had not seen a slot's tile before, the parity of the one
                // before that would look like this one's
                for (int j = 0; ok && j < tiles; ++j) {
                    const uint32_t i = it + j, sg = i % ST;
                    ok = __all_sync(0xFFFFFFFFu, wait_phase(&s.full[sg], (i / ST) & 1, &s.abort, limit));
                    if (!ok)
                        break;
                    if ((i & (kQ4Warps - 1)) == warp)
                        q4_tile<D, NQ>(st, s.ring[sg], min(kQ4Keys, u.seq.prefix - (u.tile + j) * kQ4Keys), qf, c);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&s.empty[sg]);
                }
            }
            it += tiles;
            // the next warp in turn has the nodes
            if (ok && u.tile_end == u.n_tiles && (it & (kQ4Warps - 1)) == warp) {
                Q4State<D, NQ> y = st;  // the call keeps only these copies in memory
                const AttendUnit v = u;
                q4_nodes<T, D, NQ>(a, v, y);
                st = y;
            }
            // the unit's parts of the four warps
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1)
                        st.l[q][e] += __shfl_xor_sync(0xFFFFFFFFu, st.l[q][e], k);
                    if (g == 0) {
                        s.m[warp][8 * q + 2 * t + e] = st.m[q][e];
                        s.l[warp][8 * q + 2 * t + e] = st.l[q][e];
                    }
                    float *row = s.o[warp][8 * q + 2 * t + e] + g * (D / 8);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        *reinterpret_cast<float2 *>(row + 2 * j) = make_float2(st.o[q][j][e], st.o[q][j][e + 2]);
                }
            q4_sync();
            const bool whole = u.n_parts == 1;
            float *slot = whole ? nullptr : part_slot<Sh::kRows>(a, blockIdx.x, u.part);
            for (int i = tid; i < u.n_rows * (D / 8); i += 32 * kQ4Warps) {
                const int r = i / (D / 8), d = i % (D / 8) * 8;
                float m = -INFINITY, l = 0.0f, y[8] = {}, f[kQ4Warps];
#pragma unroll
                for (int w = 0; w < kQ4Warps; ++w)
                    m = fmaxf(m, s.m[w][r]);
                const float m0 = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int w = 0; w < kQ4Warps; ++w) {
                    f[w] = exp2f(s.m[w][r] - m0);
                    l = fmaf(f[w], s.l[w][r], l);
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        const float4 z = *reinterpret_cast<const float4 *>(&s.o[w][r][d + k]);
                        y[k] = fmaf(f[w], z.x, y[k]);
                        y[k + 1] = fmaf(f[w], z.y, y[k + 1]);
                        y[k + 2] = fmaf(f[w], z.z, y[k + 2]);
                        y[k + 3] = fmaf(f[w], z.w, y[k + 3]);
                    }
                }
                const float to = whole ? (l > 0.0f || l != l ? 128.0f / l : 0.0f) : 128.0f;
                if (whole) {
                    uint4 v;
                    v.x = TcType<T>::pack(y[0] * to, y[1] * to);
                    v.y = TcType<T>::pack(y[2] * to, y[3] * to);
                    v.z = TcType<T>::pack(y[4] * to, y[5] * to);
                    v.w = TcType<T>::pack(y[6] * to, y[7] * to);
                    *reinterpret_cast<uint4 *>(reinterpret_cast<T *>(a.out) + row_place(a, u, r) + d) = v;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; k += 4)
                        __stcg(reinterpret_cast<float4 *>(slot + part_quad<Sh::kRows>((d + k) / 4, r)),
                               make_float4(y[k] * to, y[k + 1] * to, y[k + 2] * to, y[k + 3] * to));
                    if (d == 0) {
                        __stcg(slot + (size_t)Sh::kRows * D + r, m);
                        __stcg(slot + (size_t)Sh::kRows * D + Sh::kRows + r, l);
                    }
                }
            }
            if (!whole) {
                __threadfence();
                q4_sync();
                if (tid == 0) {
                    s.last = 0;
                    if (!*reinterpret_cast<volatile int *>(&s.abort)) {
                        int *cnt = part_counter(a, u.first_cta);
                        s.last = atomicAdd(cnt, 1) == u.n_parts - 1;
                        if (s.last)
                            *cnt = 0;
                    }
                }
                q4_sync();
                if (s.last) {
                    __threadfence();
                    join_parts<T, Sh::kRows>(a, u, tid, 32 * kQ4Warps, [] {
                        __threadfence();
                        q4_sync();
                        return true;
                    });
                }
            }
            q4_sync();  // the next unit's parts come after these were read
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
    const int rows = a.a.seq.T * a.a.G;
    if (rows > 16)
        return launch_attend_q4_tc(a, std::is_same<T, __half>::value ? SPEC_F16 : SPEC_BF16, st);
    if (rows <= 8)
        return launch_q4<T, D, 1>(a, st);
    return rows <= 16 ? launch_q4<T, D, 2>(a, st) : launch_q4<T, D, 3>(a, st);
}

}  // namespace

cudaError_t launch_attend_q4(const AttendQ4Args &a, spec_dtype dt, cudaStream_t st)
{
    if (a.pool.D == 64)
        return dt == SPEC_BF16 ? launch_q4_d<__nv_bfloat16, 64>(a, st) : launch_q4_d<__half, 64>(a, st);
    return dt == SPEC_BF16 ? launch_q4_d<__nv_bfloat16, 128>(a, st) : launch_q4_d<__half, 128>(a, st);
}

size_t attend_q4_workspace(int T, int Hq, int H, int D)
{
    (void)T, (void)Hq, (void)H;
    const size_t one = 2 * 3 * kAttendCtas * part_floats<8>(D), many = 2 * 2 * kAttendCtas * part_floats<24>(D);
    const size_t few = align256(kPartHead + (one > many ? one : many) * sizeof(float)), tc = attend_q4_tc_workspace(D);
    return few > tc ? few : tc;
}

}  // namespace spec
