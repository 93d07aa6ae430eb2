// append.cu -- the fused projection's queries, keys and values of a round or
// a prompt, taken to where attention reads them, in one pass.
//
// For each token and each query and key head x[0..D):
//   y = x * rsqrt(mean(x^2) + eps) * w            (w null: y = x)
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = pos * inv_freq[i]
// over the pairs j = i + R/2 (or (2i, 2i + 1) when interleaved); dimensions
// past R are not turned.  Everything between the load and the store is fp32,
// rounded once.  Values are copied.  The angle is a product of an integer
// position and an fp32 frequency whose turns are what matters: it is formed
// and reduced in fp64 (a position of 1e5 in fp32 would be off by 4e-3 turns),
// once per token and pair, not per head.
//
// Roofline: HBM, 2 * (Hq + 2H) * D * sizeof(T) bytes per token.
#include "forward.h"
#include "spec_common.cuh"

namespace spec {

constexpr int kAppendThreads = 256;
constexpr int kAppendAhead = 4;  // 16-byte loads of a thread in flight before the angles are ready

// round-to-nearest stores of fp32 values
template <typename T>
__device__ __forceinline__ T to_storage(float x);
template <>
__device__ __forceinline__ float to_storage<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_storage<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half to_storage<__half>(float x) { return __float2half_rn(x); }

template <typename T>
__device__ __forceinline__ uint4 pack16(const float *f)
{
    constexpr int VEC = Storage<T>::kVec;
    T t[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        t[i] = to_storage<T>(f[i]);
    uint4 u;
    memcpy(&u, t, 16);
    return u;
}

// The token of this CTA: its sequence, place and position.
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

__device__ Token find_token(const AppendArgs &a, long long m)
{
    Token t;
    t.live = false;
    t.q_row = m;
    int b, i;
    if (a.seq.cu) {
        // the sequences that end at or before m come before m's: counted by
        // each warp in one pass over cu, which also looks at its order
        const int lane = threadIdx.x & 31;
        int before = 0;
        unsigned broken = 0;
        for (int c = 0; c < a.seq.B; c += 32) {
            const bool in = c + lane < a.seq.B;
            const int lo = in ? a.seq.cu[c + lane] : 0, hi = in ? a.seq.cu[c + lane + 1] : 0;
            before += __popc(__ballot_sync(0xFFFFFFFFu, in && hi <= m));
            broken |= __ballot_sync(0xFFFFFFFFu, hi < lo);
        }
        b = before;
        if (b >= a.seq.B || broken)
            return t;
    } else {
        b = (int)(m / a.seq.T);
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

__device__ void append_flags(const AppendArgs &a)
{
    if (blockIdx.x != 0 || !a.flags)
        return;
    bool broken = false;  // packed offsets that descend anywhere: no sequence of the call is taken
    if (a.seq.cu) {
        for (int b = threadIdx.x; b < a.seq.B; b += blockDim.x)
            broken |= a.seq.cu[b + 1] < a.seq.cu[b];
        broken = __syncthreads_or(broken);
    }
    for (int b = threadIdx.x; b < a.seq.B; b += blockDim.x)
        a.flags[b] = !broken && load_seq(a.seq, a.cache.N, a.cache.S, b).ok ? 0u : SPEC_FLAG_BAD_STATE;
    if (a.seq.idx && writes_cache(a.seq)) {
        __syncthreads();
        for (int b = threadIdx.x >> 5; b < a.seq.B; b += blockDim.x >> 5) {  // warp-uniform
            const bool twice = repeated_row(a.seq.idx, a.seq.B, a.seq.idx[b]);
            if (twice && (threadIdx.x & 31) == 0)
                a.flags[b] = SPEC_FLAG_BAD_STATE;
        }
    }
}

// cos and sin of pos * f.  The turns left after reduction are exact to fp64;
// the fp32 argument's rounding is put back to first order.
__device__ __forceinline__ float2 turn(int pos, float f)
{
    double t = (double)pos * (double)f * 0.15915494309189533577;  // 1 / (2 pi)
    t = 2.0 * (t - rint(t));  // half turns in [-1, 1]
    const float h = (float)t;
    const float d = (float)(t - (double)h) * 3.14159265358979f;
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

// One CTA per token; LPH lanes hold one head, 16 bytes each.  Rotation over
// the whole head (R == D) or none.  A thread's first kAppendAhead heads are
// loaded before the angles are computed.
template <typename T, int LPH>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a)
{
    constexpr int VEC = Storage<T>::kVec;
    constexpr int D = LPH * VEC;
    constexpr int GROUPS = kAppendThreads / LPH;
    __shared__ float2 s_turn[D / 2];
    append_flags(a);
    const Token tok = find_token(a, blockIdx.x);
    if (!tok.live)
        return;
    const int heads = a.Hq + 2 * a.cache.H;
    const int grp = threadIdx.x / LPH, ln = threadIdx.x % LPH;
    const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.qkv) + tok.q_row * heads * D) + ln;
    for (int base = 0; base < heads; base += GROUPS * kAppendAhead) {
        uint4 r[kAppendAhead];
#pragma unroll
        for (int u = 0; u < kAppendAhead; ++u) {
            const int head = base + u * GROUPS + grp;
            if (head < heads)
                r[u] = ld_stream16(src + (size_t)head * LPH);
        }
        if (base == 0 && a.R) {
            for (int i = threadIdx.x; i < D / 2; i += kAppendThreads)
                s_turn[i] = turn(tok.pos, a.inv_freq[i]);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kAppendAhead; ++u) {
            const int head = base + u * GROUPS + grp;
            // warps stay whole up to here: the shuffles below need every lane
            if (base + u * GROUPS >= heads)
                break;
            const bool mine = head < heads;
            const bool is_v = head >= a.Hq + a.cache.H;
            float x[VEC];
            Storage<T>::unpack(r[u], x);
            if (!mine) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    x[e] = 0.0f;
            }
            const T *w = reinterpret_cast<const T *>(head < a.Hq ? a.q_weight : a.k_weight);
            if (a.q_weight || a.k_weight) {  // the same for every thread
                float sq = 0.0f;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    sq = fmaf(x[e], x[e], sq);
#pragma unroll
                for (int m = LPH / 2; m > 0; m >>= 1)
                    sq += __shfl_xor_sync(0xFFFFFFFFu, sq, m);
                if (w && !is_v) {
                    const float inv = rsqrtf(sq * (1.0f / D) + a.eps);
                    float g[VEC];
                    Storage<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(w) + ln), g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        x[e] = x[e] * inv * g[e];
                }
            }
            if (a.R) {
                if (a.interleaved) {
                    if (!is_v) {
#pragma unroll
                        for (int e = 0; e < VEC; e += 2) {
                            const float2 cs = s_turn[(ln * VEC + e) / 2];
                            const float lo = x[e], hi = x[e + 1];
                            x[e] = lo * cs.x - hi * cs.y;
                            x[e + 1] = hi * cs.x + lo * cs.y;
                        }
                    }
                } else {
                    // the other half of each pair is LPH / 2 lanes away
                    const bool low = ln < LPH / 2;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float o = __shfl_xor_sync(0xFFFFFFFFu, x[e], LPH / 2);
                        if (!is_v) {
                            const float2 cs = s_turn[(ln % (LPH / 2)) * VEC + e];
                            x[e] = low ? x[e] * cs.x - o * cs.y : x[e] * cs.x + o * cs.y;
                        }
                    }
                }
            }
            if (mine)
                reinterpret_cast<uint4 *>(head_dst<T>(a, tok, head))[ln] = is_v ? r[u] : pack16<T>(x);
        }
    }
}

// Any head size and any R <= D: one warp per head, the head in shared memory.
constexpr int kMaxHeadDim = SPEC_MAX_HEAD_DIM;
template <typename T>
__global__ void __launch_bounds__(kAppendThreads) append_any_kernel(AppendArgs a)
{
    __shared__ float s_x[kAppendThreads / 32][kMaxHeadDim];
    __shared__ float2 s_turn[kMaxHeadDim / 2];
    append_flags(a);
    const Token tok = find_token(a, blockIdx.x);
    if (!tok.live)
        return;
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
}

template <typename T>
cudaError_t launch_append_t(const AppendArgs &a, cudaStream_t st)
{
    const unsigned grid = (unsigned)(a.seq.cu ? (a.seq.M > 0 ? a.seq.M : 1) : a.seq.B * a.seq.T);
    const int D = a.cache.D;
    const long long bytes = (long long)D * sizeof(T);
    auto ok16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool vec = (a.R == D || a.R == 0) && ok16(a.qkv) && ok16(a.q_out) && ok16(a.kv_out) && ok16(a.staged) &&
                     ok16(a.q_weight) && ok16(a.k_weight);
    if (vec && bytes == 512)
        append_kernel<T, 32><<<grid, kAppendThreads, 0, st>>>(a);
    else if (vec && bytes == 256)
        append_kernel<T, 16><<<grid, kAppendThreads, 0, st>>>(a);
    else if (vec && bytes == 128)
        append_kernel<T, 8><<<grid, kAppendThreads, 0, st>>>(a);
    else
        append_any_kernel<T><<<grid, kAppendThreads, 0, st>>>(a);
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
