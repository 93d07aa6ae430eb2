// append.cu -- the fused projection's queries, keys and values of a round or
// a prompt, taken to where attention reads them, in one pass.
//
// For each token and each query and key head x[0..D):
//   y = x * rsqrt(mean(x^2) + eps) * w            (w null: y = x)
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = pos * inv_freq[i]
// over the pairs j = i + R/2 (or (2i, 2i + 1) when interleaved); dimensions
// past R are not turned.  Everything between the load and the store is fp32,
// rounded once.  Values are copied.  The angle is a product of an integer
// position and an fp32 frequency, of which the fraction of its turns matters: it
// is reduced to that by `turn` (rounded to fp32 as it is, a position of 1e5
// would be off by 6e-4 turns), once per token and pair, not per head.
//
// Roofline: HBM, 2 * (Hq + 2H) * D * sizeof(T) bytes per token.
#include "forward.h"
#include "packed.cuh"
#include "spec_common.cuh"

namespace spec {

constexpr int kAppendThreads = 128;
constexpr int kAppendAhead = 4;     // heads of a thread whose loads are in flight together
constexpr int kAppendWarps = 2432;  // with fewer warps than this (16 an SM) tokens are shared out

// round-to-nearest stores of fp32 values
template <typename T>
__device__ __forceinline__ T to_storage(float x);
template <>
__device__ __forceinline__ float to_storage<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_storage<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half to_storage<__half>(float x) { return __float2half_rn(x); }

// A token: its sequence, place and position.
struct Token {
    bool live;
    long long q_row;  // row of qkv and q_out
    long long kv_off; // element offset of (head 0, this token) in the K slabs' base, heads head_step apart
    long long head_step;
    bool to_staged;
    int pos;
};

// staged nodes are written by sequence, so a repeated cache row only matters
// to the calls that write the cache
__device__ __forceinline__ bool writes_cache(const SeqArgs &s) { return !s.staged; }

// by a whole warp
__device__ Token find_token(const AppendArgs &a, long long m)
{
    Token t;
    t.live = false;
    t.q_row = m;
    int b, i;
    if (a.seq.cu) {
        // the sequences that end at or before m come before m's: counted by
        // each warp in one pass over cu, which also looks at its order (the
        // lanes' counts meet at the end, so that the loads need not wait for
        // one another)
        int before = 0;
        bool broken = false;
#pragma unroll 8
        for (int c = threadIdx.x & 31; c < a.seq.B; c += 32) {
            const int lo = a.seq.cu[c], hi = a.seq.cu[c + 1];
            before += hi <= m;
            broken |= hi < lo;
        }
        b = __reduce_add_sync(0xFFFFFFFFu, before);
        if (b >= a.seq.B || __any_sync(0xFFFFFFFFu, broken))
            return t;
    } else {
        b = (int)((uint32_t)m / (uint32_t)a.seq.T);
    }
    const Seq s = load_seq(a.seq, a.cache.N, a.cache.S, b);
    i = (int)(m - s.tok0);
    if (!s.ok || i < 0 || i >= s.n || (writes_cache(a.seq) && repeated_row(a.seq.idx, a.seq.B, s.row)))
        return t;
    t.live = true;
    const int dep = a.depth ? a.depth[(size_t)b * a.seq.T + i] : i;
    t.pos = s.prefix + dep;
    const long long D = a.cache.D;
    if (a.seq.staged) {
        t.to_staged = true;
        t.head_step = (long long)a.seq.T * D;
        t.kv_off = ((long long)b * a.cache.H * a.seq.T + i) * D;
    } else {
        t.to_staged = false;
        t.head_step = (long long)a.cache.S * D;
        t.kv_off = ((long long)s.row * a.cache.H * a.cache.S + s.slot0 + s.prefix + i) * D;
    }
    return t;
}

// Flags, sequence b's by warp b of the grid and so on around, after its token:
// a repeated row costs a look at every sequence's, which one CTA would do B
// times over.  By whole warps.
__device__ void append_flags(const AppendArgs &a)
{
    if (!a.flags)
        return;
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
    long long b = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (b >= a.seq.B)
        return;
    bool broken = false;  // packed offsets that descend anywhere: no sequence of the call is taken
    if (a.seq.cu) {
        for (int c = lane; c < a.seq.B; c += 32)
            broken |= a.seq.cu[c + 1] < a.seq.cu[c];
        broken = __any_sync(0xFFFFFFFFu, broken);
    }
    for (; b < a.seq.B; b += warps) {
        bool ok = !broken && load_seq(a.seq, a.cache.N, a.cache.S, (int)b).ok;
        if (a.seq.idx && writes_cache(a.seq))
            ok = !repeated_row(a.seq.idx, a.seq.B, a.seq.idx[b]) && ok;
        if (lane == 0)
            a.flags[b] = ok ? 0u : SPEC_FLAG_BAD_STATE;
    }
}

// cos and sin of pos * f.  Only the fraction of pos * f / (2 pi) turns counts.
// f / (2 pi) is a pair g + gl of fp32 numbers (48 bits); pos * g is split by an
// FMA into its rounded value t, whose fraction is exact, and the rest e, and the
// sum of the two keeps what its rounding leaves off (d).  For |pos * f| < 2^22,
// and below 2^24 where an fp32 pos is exact, the error is then that of 48 bits
// at 2^22 / (2 pi) turns: under 1e-8 turns.  Past either limit the same in fp64
// (two lanes a clock on this part, 10 times the time), with an error below that
// of the result's last place.
__device__ __forceinline__ float2 turn(int pos, float f)
{
    float h, d;  // half turns in [-1, 1], and what its rounding left off, in radians
    constexpr float kPi = 3.14159265358979f;
    const float p = (float)pos;
    if (pos < (1 << 24) && fabsf(p * f) < 4194304.0f) {
        constexpr float kHi = 0.15915493667125702f, kLo = 6.420638243e-09f;  // 1 / (2 pi)
        const float g = f * kHi, gl = fmaf(f, kHi, -g) + f * kLo;
        const float t = p * g, e = fmaf(p, g, -t) + p * gl;
        const float a = t - rintf(t), s = a + e, b = s - a;
        h = 2.0f * (s - rintf(s));
        d = 2.0f * kPi * ((a - (s - b)) + (e - b));
    } else {
        constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
        const double x = pos, y = f, z = x * y;
        const double t = z * kHi, e = fma(z, kHi, -t) + (z * kLo + fma(x, y, -z) * kHi);
        double r = (t - rint(t)) + e;
        r = 2.0 * (r - rint(r));
        h = (float)r;
        d = (float)(r - (double)h) * kPi;
    }
    float s, c;
    sincospif(h, &s, &c);
    return make_float2(fmaf(-s, d, c), fmaf(c, d, s));
}

// destination of head `head`'s element 0: queries, keys, then values
template <typename T>
__device__ __forceinline__ T *head_dst(const AppendArgs &a, const Token &t, int head)
{
    const int D = a.cache.D, H = a.cache.H;
    if (head < a.Hq)
        return reinterpret_cast<T *>(a.q_out) + (t.q_row * a.Hq + head) * D;
    const bool is_v = head >= a.Hq + H;
    const int h = head - a.Hq - (is_v ? H : 0);
    const long long row_len = (long long)(t.to_staged ? a.seq.T : a.cache.S) * D;
    T *base = reinterpret_cast<T *>(t.to_staged ? a.staged : a.kv_out);
    const long long slab = t.to_staged ? (is_v ? a.st_v : a.st_k) : (is_v ? a.cache.v_slab : a.cache.k_slab);
    return base + slab * row_len + t.kv_off + h * t.head_step;
}

// 8 bytes of storage as fp32 pairs (one for fp32, two for 16-bit types)
template <typename T>
struct Half8;
template <>
struct Half8<float> {
    static constexpr int kPairs = 1;
    __device__ static void load(uint2 u, uint64_t *x) { x[0] = pair(__uint_as_float(u.x), __uint_as_float(u.y)); }
    __device__ static uint2 store(const uint64_t *x)
    {
        const float2 f = unpair(x[0]);
        return make_uint2(__float_as_uint(f.x), __float_as_uint(f.y));
    }
};
template <>
struct Half8<__nv_bfloat16> {
    static constexpr int kPairs = 2;
    __device__ static uint64_t word(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
    __device__ static void load(uint2 u, uint64_t *x)
    {
        x[0] = word(u.x);
        x[1] = word(u.y);
    }
    __device__ static uint32_t back(uint64_t x)
    {
        const float2 f = unpair(x);
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
        return r;
    }
    __device__ static uint2 store(const uint64_t *x) { return make_uint2(back(x[0]), back(x[1])); }
};
template <>
struct Half8<__half> {
    static constexpr int kPairs = 2;
    __device__ static uint64_t word(uint32_t w)
    {
        __half2 h;
        memcpy(&h, &w, 4);
        const float2 f = __half22float2(h);
        return pair(f.x, f.y);
    }
    __device__ static void load(uint2 u, uint64_t *x)
    {
        x[0] = word(u.x);
        x[1] = word(u.y);
    }
    __device__ static uint32_t back(uint64_t x)
    {
        const float2 f = unpair(x);
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
        return r;
    }
    __device__ static uint2 store(const uint64_t *x) { return make_uint2(back(x[0]), back(x[1])); }
};

__device__ __forceinline__ uint2 ld_stream8(const uint2 *p)
{
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// Both kernels below: LPH lanes hold one head, 8 bytes of its first half and
// the same 8 of its second, so that a rotation's pairs are in one lane, as are
// the angles and norm weights of all heads of a token.  Rotation over the whole
// head (R == D) or none.  The first loads are asked for before anything else:
// what decides the token's place and angles is a chain of three loads itself.
// 26624 tokens of 48 heads of 128 in bf16, where HBM needs 96 us: a first form
// with a CTA a token and 16 contiguous bytes a lane (8 shuffles a vector for the
// pairs, angles and weights from shared memory) took 216, a warp a token with
// all kinds of heads in one loop 129 (an issue slot in two was taken), this
// split 105 (6.2 TB/s).  What bounds it is the loads in flight and what issues
// between them: 2, 3 or 8 loads ahead instead of 4 measured 117, 114 and 110, 72
// registers instead of 64 (7 CTAs instead of 8) 107.

// cosines, sines and minus sines of a lane's pairs.  Half split: pair i of the
// lane turns with frequency 2 NP ln + i; interleaved: elements (2 i, 2 i + 1)
// of each half with NP ln + i and D / 4 + NP ln + i
template <int NP, int D>
__device__ __forceinline__ void turns(const AppendArgs &a, int pos, int ln, uint64_t *cs, uint64_t *sn, uint64_t *ns)
{
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int f0 = a.interleaved ? NP * ln + i : 2 * NP * ln + 2 * i;
        const int f1 = a.interleaved ? D / 4 + NP * ln + i : f0 + 1;
        const float2 t0 = turn(pos, a.inv_freq[f0]), t1 = turn(pos, a.inv_freq[f1]);
        cs[i] = pair(t0.x, t1.x);
        sn[i] = pair(t0.y, t1.y);
        ns[i] = pair(-t0.y, -t1.y);
    }
}
// sum of the squares of a head, in each of its LPH lanes
template <int NP, int LPH>
__device__ __forceinline__ float square_sum(const uint64_t *x)
{
    uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 2 * NP; ++i)
        sq = fma2(x[i], x[i], sq);
    const float2 q2 = unpair(sq);
    float sum = q2.x + q2.y;
#pragma unroll
    for (int k = LPH / 2; k > 0; k >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
    return sum;
}
template <int NP>
__device__ __forceinline__ void scale(float inv, uint64_t *x, const uint64_t *g)
{
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i)
        x[i] = mul2(mul2(x[i], pair(inv, inv)), g[i]);
}
template <int NP, int LPH, int D>
__device__ __forceinline__ void norm(float eps, uint64_t *x, const uint64_t *g)
{
    scale<NP>(rsqrtf(square_sum<NP, LPH>(x) * (1.0f / D) + eps), x, g);
}
template <int NP>
__device__ __forceinline__ void rotate(int interleaved, uint64_t *x, const uint64_t *cs, const uint64_t *sn,
                                       const uint64_t *ns)
{
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        if (!interleaved) {
            const uint64_t l = x[i], h = x[NP + i];
            x[i] = fma2(l, cs[i], mul2(h, ns[i]));
            x[NP + i] = fma2(h, cs[i], mul2(l, sn[i]));
        } else {
            const float2 c = unpair(cs[i]), s = unpair(sn[i]), l = unpair(x[i]), h = unpair(x[NP + i]);
            x[i] = pair(l.x * c.x - l.y * s.x, l.y * c.x + l.x * s.x);
            x[NP + i] = pair(h.x * c.y - h.y * s.y, h.y * c.y + h.x * s.y);
        }
    }
}

// `share` warps per token, where there are not tokens enough to fill the GPU
// with one each (2 to 8); all kinds of heads in one loop, as a warp has few.
// 36 heads of 128, shared out against a warp a token: 64 tokens 3.8 us, 7.3; 288
// tokens 4.1, 7.4; 832 tokens 7.0, 8.0; with up to 9728 warps, the other way
// round, 4096 tokens took 21.6 instead of 14.0.
template <typename T, int LPH>
__device__ __forceinline__ void append_token(const AppendArgs &a, int tokens, int share)
{
    using H8 = Half8<T>;
    constexpr int NP = H8::kPairs;                 // pairs of elements in 8 bytes
    constexpr int D = LPH * 16 / (int)sizeof(T);
    constexpr int HPW = 32 / LPH;                  // heads a warp holds at a time
    const int lane = threadIdx.x & 31, ln = lane % LPH;
    const uint32_t gw = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const uint32_t m = gw / (uint32_t)share;
    if (m >= (uint32_t)tokens)
        return;
    const int heads = a.Hq + 2 * a.cache.H;
    const int first = (int)(gw - m * (uint32_t)share) * HPW + lane / LPH, step = share * HPW;
    const T *src = reinterpret_cast<const T *>(a.qkv) + (size_t)m * heads * D + ln * 2 * NP;
    Token tok;
    T *q0, *k0, *v0;                               // head 0 of each kind
    uint64_t cs[NP], sn[NP], ns[NP];               // per pair of elements: cosines, sines, minus sines
    uint64_t gq[NP * 2], gk[NP * 2];
    for (int base = 0; base < heads; base += kAppendAhead * step) {
        uint2 lo[kAppendAhead], hi[kAppendAhead];
#pragma unroll
        for (int u = 0; u < kAppendAhead; ++u) {
            const int head = base + u * step + first;
            if (head < heads) {
                lo[u] = ld_stream8(reinterpret_cast<const uint2 *>(src + (long long)head * D));
                hi[u] = ld_stream8(reinterpret_cast<const uint2 *>(src + (long long)head * D + D / 2));
            }
        }
        if (base == 0) {
            auto weights = [&](const void *w, uint64_t *g) {
                const T *p = reinterpret_cast<const T *>(w) + ln * 2 * NP;
                H8::load(__ldg(reinterpret_cast<const uint2 *>(p)), g);
                H8::load(__ldg(reinterpret_cast<const uint2 *>(p + D / 2)), g + NP);
            };
            if (a.q_weight)
                weights(a.q_weight, gq);
            if (a.k_weight)
                weights(a.k_weight, gk);
            tok = find_token(a, m);
            if (!tok.live)
                return;  // the whole warp
            q0 = head_dst<T>(a, tok, 0) + ln * 2 * NP;
            k0 = head_dst<T>(a, tok, a.Hq) + ln * 2 * NP;
            v0 = head_dst<T>(a, tok, a.Hq + a.cache.H) + ln * 2 * NP;
            if (a.R)
                turns<NP, D>(a, tok.pos, ln, cs, sn, ns);
        }
#pragma unroll
        for (int u = 0; u < kAppendAhead; ++u) {
            if (base + u * step >= heads)
                break;  // the warp stays whole for the shuffles
            const int head = base + u * step + first;
            const bool mine = head < heads, is_v = head >= a.Hq + a.cache.H;
            uint2 ol = lo[u], oh = hi[u];
            if (__any_sync(0xFFFFFFFFu, mine && !is_v)) {
                uint64_t x[2 * NP];
                H8::load(mine ? lo[u] : make_uint2(0, 0), x);
                H8::load(mine ? hi[u] : make_uint2(0, 0), x + NP);
                const bool is_q = head < a.Hq;
                if (a.q_weight || a.k_weight) {  // the same for every thread
                    const float sum = square_sum<NP, LPH>(x);
                    if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr)
                        scale<NP>(rsqrtf(sum * (1.0f / D) + a.eps), x, is_q ? gq : gk);
                }
                if (a.R)
                    rotate<NP>(a.interleaved, x, cs, sn, ns);
                if (!is_v) {
                    ol = H8::store(x);
                    oh = H8::store(x + NP);
                }
            }
            if (mine) {
                T *dst = head < a.Hq ? q0 + head * D : (is_v ? v0 : k0) + (head - a.Hq - (is_v ? a.cache.H : 0)) * tok.head_step;
                *reinterpret_cast<uint2 *>(dst) = ol;
                *reinterpret_cast<uint2 *>(dst + D / 2) = oh;
            }
        }
    }
}

// A warp a token, the heads of a kind after one another: what a head is, its
// weights and where it goes are then the same for the whole warp.
template <typename T, int LPH>
__device__ __forceinline__ void append_whole_token(const AppendArgs &a, int tokens)
{
    using H8 = Half8<T>;
    constexpr int NP = H8::kPairs, D = LPH * 16 / (int)sizeof(T), HPW = 32 / LPH, UP = kAppendAhead;
    const int lane = threadIdx.x & 31, ln = lane % LPH, sub = lane / LPH;
    const uint32_t m = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (m >= (uint32_t)tokens)
        return;
    const int H = a.cache.H;
    const T *src = reinterpret_cast<const T *>(a.qkv) + ((size_t)m * (a.Hq + 2 * H) + sub) * D + ln * 2 * NP;
    uint2 lo[UP], hi[UP];
    // heads at + u HPW + sub of the n from p on
    auto load = [&](const T *p, int at, int n) {
#pragma unroll
        for (int u = 0; u < UP; ++u)
            if (at + u * HPW + sub < n) {
                lo[u] = ld_stream8(reinterpret_cast<const uint2 *>(p + (size_t)at * D + u * HPW * D));
                hi[u] = ld_stream8(reinterpret_cast<const uint2 *>(p + (size_t)at * D + u * HPW * D + D / 2));
            }
    };
    load(src, 0, a.Hq);
    uint64_t g[NP * 2];
    auto weights = [&](const void *w) {
        const T *p = reinterpret_cast<const T *>(w) + ln * 2 * NP;
        H8::load(__ldg(reinterpret_cast<const uint2 *>(p)), g);
        H8::load(__ldg(reinterpret_cast<const uint2 *>(p + D / 2)), g + NP);
    };
    if (a.q_weight)
        weights(a.q_weight);
    const Token tok = find_token(a, m);
    if (!tok.live)
        return;  // the whole warp
    uint64_t cs[NP], sn[NP], ns[NP];
    if (a.R)
        turns<NP, D>(a, tok.pos, ln, cs, sn, ns);
    auto turn_store = [&](T *dst, long long head_step, int at, int n, const void *w) {
        dst += ln * 2 * NP + (at + sub) * head_step;
#pragma unroll
        for (int u = 0; u < UP; ++u) {
            if (at + u * HPW >= n)
                break;
            uint64_t x[2 * NP];
            H8::load(lo[u], x);
            H8::load(hi[u], x + NP);
            if (w)
                norm<NP, LPH, D>(a.eps, x, g);
            if (a.R)
                rotate<NP>(a.interleaved, x, cs, sn, ns);
            if (at + u * HPW + sub < n) {
                T *d = dst + u * HPW * head_step;
                *reinterpret_cast<uint2 *>(d) = H8::store(x);
                *reinterpret_cast<uint2 *>(d + D / 2) = H8::store(x + NP);
            }
        }
    };
    T *q0 = head_dst<T>(a, tok, 0), *k0 = head_dst<T>(a, tok, a.Hq), *v0 = head_dst<T>(a, tok, a.Hq + H);
    for (int at = 0;;) {
        turn_store(q0, D, at, a.Hq, a.q_weight);
        at += UP * HPW;
        if (at >= a.Hq)
            break;
        load(src, at, a.Hq);
    }
    src += (size_t)a.Hq * D;
    load(src, 0, H);
    if (a.k_weight)
        weights(a.k_weight);
    for (int at = 0;;) {
        turn_store(k0, tok.head_step, at, H, a.k_weight);
        at += UP * HPW;
        if (at >= H)
            break;
        load(src, at, H);
    }
    src += (size_t)H * D;
    for (int at = 0; at < H; at += UP * HPW) {
        load(src, at, H);
        T *dst = v0 + ln * 2 * NP + (at + sub) * tok.head_step;
#pragma unroll
        for (int u = 0; u < UP; ++u)
            if (at + u * HPW + sub < H) {
                *reinterpret_cast<uint2 *>(dst + u * HPW * tok.head_step) = lo[u];
                *reinterpret_cast<uint2 *>(dst + u * HPW * tok.head_step + D / 2) = hi[u];
            }
    }
}

template <typename T, int LPH>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a, int tokens,
                                                                int share)
{
    append_token<T, LPH>(a, tokens, share);
    append_flags(a);
}
template <typename T, int LPH>
__global__ void __launch_bounds__(kAppendThreads, 8) append_whole_kernel(const __grid_constant__ AppendArgs a, int tokens)
{
    append_whole_token<T, LPH>(a, tokens);
    append_flags(a);
}

// Any head size and any R <= D: one warp per head, the head in shared memory.
constexpr int kMaxHeadDim = SPEC_MAX_HEAD_DIM;
template <typename T>
__global__ void __launch_bounds__(kAppendThreads) append_any_kernel(const __grid_constant__ AppendArgs a)
{
    __shared__ float s_x[kAppendThreads / 32][kMaxHeadDim];
    __shared__ float2 s_turn[kMaxHeadDim / 2];
    const Token tok = a.seq.M || !a.seq.cu ? find_token(a, blockIdx.x) : Token{};
    if (!tok.live) {  // the whole CTA
        append_flags(a);
        return;
    }
    const int D = a.cache.D, half = a.R / 2;
    for (int i = threadIdx.x; i < half; i += kAppendThreads)
        s_turn[i] = turn(tok.pos, a.inv_freq[i]);
    __syncthreads();
    const int heads = a.Hq + 2 * a.cache.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *x = s_x[warp];
    for (int head = warp; head < heads; head += kAppendThreads / 32) {
        const T *src = reinterpret_cast<const T *>(a.qkv) + (tok.q_row * heads + head) * D;
        T *dst = head_dst<T>(a, tok, head);
        if (head >= a.Hq + a.cache.H) {
            for (int d = lane; d < D; d += 32)
                dst[d] = src[d];
            continue;
        }
        float sq = 0.0f;
        for (int d = lane; d < D; d += 32) {
            x[d] = Storage<T>::at(src, d);
            sq = fmaf(x[d], x[d], sq);
        }
        const T *w = reinterpret_cast<const T *>(head < a.Hq ? a.q_weight : a.k_weight);
        if (w) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1)
                sq += __shfl_xor_sync(0xFFFFFFFFu, sq, m);
            const float inv = rsqrtf(sq / D + a.eps);
            for (int d = lane; d < D; d += 32)
                x[d] = x[d] * inv * Storage<T>::at(w, d);
        }
        __syncwarp();
        for (int i = lane; i < half; i += 32) {
            const int p = a.interleaved ? 2 * i : i, q = a.interleaved ? 2 * i + 1 : i + half;
            const float2 cs = s_turn[i];
            const float lo = x[p], hi = x[q];
            dst[p] = to_storage<T>(lo * cs.x - hi * cs.y);
            dst[q] = to_storage<T>(hi * cs.x + lo * cs.y);
        }
        for (int d = a.R + lane; d < D; d += 32)
            dst[d] = to_storage<T>(x[d]);
        __syncwarp();
    }
    append_flags(a);
}

template <typename T>
cudaError_t launch_append_t(const AppendArgs &a, cudaStream_t st)
{
    const int tokens = a.seq.cu ? a.seq.M : a.seq.B * a.seq.T;
    const int D = a.cache.D;
    const long long bytes = (long long)D * sizeof(T);
    auto ok16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool vec = (a.R == D || a.R == 0) && ok16(a.qkv) && ok16(a.q_out) && ok16(a.kv_out) && ok16(a.staged) &&
                     ok16(a.q_weight) && ok16(a.k_weight);
    if (vec && (bytes == 512 || bytes == 256 || bytes == 128)) {
        int share = 1;
        while (share < 8 && (long long)tokens * share * 2 <= kAppendWarps)
            share *= 2;
        const long long warps = (long long)tokens * share, per = kAppendThreads / 32;
        const unsigned grid = (unsigned)(warps > 0 ? (warps + per - 1) / per : 1);
        if (share == 1) {
            if (bytes == 512)
                append_whole_kernel<T, 32><<<grid, kAppendThreads, 0, st>>>(a, tokens);
            else if (bytes == 256)
                append_whole_kernel<T, 16><<<grid, kAppendThreads, 0, st>>>(a, tokens);
            else
                append_whole_kernel<T, 8><<<grid, kAppendThreads, 0, st>>>(a, tokens);
        } else if (bytes == 512)
            append_kernel<T, 32><<<grid, kAppendThreads, 0, st>>>(a, tokens, share);
        else if (bytes == 256)
            append_kernel<T, 16><<<grid, kAppendThreads, 0, st>>>(a, tokens, share);
        else
            append_kernel<T, 8><<<grid, kAppendThreads, 0, st>>>(a, tokens, share);
    } else {
        append_any_kernel<T><<<(unsigned)(tokens > 0 ? tokens : 1), kAppendThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs &a, spec_dtype dt, cudaStream_t st)
{
    switch (dt) {
    case SPEC_F32:
        return launch_append_t<float>(a, st);
    case SPEC_BF16:
        return launch_append_t<__nv_bfloat16>(a, st);
    default:
        return launch_append_t<__half>(a, st);
    }
}

}  // namespace spec
