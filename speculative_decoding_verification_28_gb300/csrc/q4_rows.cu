// q4_rows.cu -- rows of 16-bit keys and values stored into pages of 4-bit codes,
// and loaded back.
//
// Each group of 32 values is read once and written once: 2 D + 17 D / 32 bytes a
// row, so HBM bounds both; a thread's group needs no other thread.  The
// products and quotients are exact (q4.cuh), so any order gives the same bytes.
#include "paged.h"
#include "q4_expand.cuh"

namespace spec {

constexpr int kRowThreads = 128;
constexpr int kRowTokens = 64;  // tokens of a CTA
constexpr int kRowSlabs = 8;    // (layer, K or V, head) slabs of a CTA

// What a CTA knows of its sequence's tokens t0 .. t0 + m - 1.
struct RowTile {
    int m;
    int at[kRowTokens];        // row within a slab of it, or -1: left out
    int page[kRowTokens];
    short in_page[kRowTokens];
    long long in_pool[kRowSlabs];  // first block of page 0 of a (layer, K or V, head), in bytes
    long long in_rows[kRowSlabs];  // and the slab of the 16-bit block, in elements
};

// Checks sequence b, fills the tile; false: nothing to do.  The CTAs of token
// tile 0 and slab 0 write the flags.
template <bool STORE>
__device__ bool row_tile(const Q4RowsArgs &a, RowTile &s)
{
    const int b = blockIdx.y, t0 = blockIdx.x * kRowTokens;
    const PoolView &v = a.pool;
    const int n = a.count[b], pos = a.pos[b], slot = a.slot ? a.slot[b] : 0;
    const int from = a.idx ? a.idx[b] : b, trow = a.row ? a.row[b] : b;
    const int page = 1 << v.page_log2;
    bool ok = n >= 0 && n <= a.T && pos >= 0 && (long long)pos + n <= (long long)v.MP * page && slot >= 0 && from >= 0 &&
              from < a.N && trow >= 0 && trow < v.R;
    ok = ok && (a.path || (long long)slot + n <= a.S);
    // after a reservation that came short, rows may share the pages that they were to write
    ok = ok && !(STORE && a.missing && *a.missing != 0);
    // sequences that write the same rows
    const bool twice = STORE ? repeated_row(a.row, a.B, trow) : repeated_row(a.idx, a.B, from);
    bool fits = true;
    if (ok && a.path)
        for (int j = threadIdx.x; j < n; j += kRowThreads) {
            const long long p = (long long)a.path[(size_t)b * a.T + j];
            fits &= p >= 0 && slot + p < a.S;
        }
    const bool first = blockIdx.x == 0 && blockIdx.z == 0 && a.flags;
    ok = __syncthreads_and(ok && !twice && fits);
    if (first) {
        bool pages = true;
        if (ok && n > 0)
            for (int p = (pos >> v.page_log2) + threadIdx.x; p <= (pos + n - 1) >> v.page_log2; p += kRowThreads) {
                const int at = v.table[(size_t)trow * v.MP + p];
                pages &= at >= 0 && at < v.P;
            }
        pages = __syncthreads_and(pages);
        if (threadIdx.x == 0)
            a.flags[b] = ok && pages ? 0u : SPEC_FLAG_BAD_STATE;
    }
    if (!ok || t0 >= n)
        return false;
    const int m = min(kRowTokens, n - t0);
    for (int j = threadIdx.x; j < m; j += kRowThreads) {
        const int p = pos + t0 + j;
        const int at = v.table[(size_t)trow * v.MP + (p >> v.page_log2)];
        const bool in = at >= 0 && at < v.P;
        s.page[j] = in ? at : 0;
        s.in_page[j] = (short)(p & (page - 1));
        s.at[j] = in ? slot + (a.path ? a.path[(size_t)b * a.T + t0 + j] : t0 + j) : -1;
    }
    if (threadIdx.x < kRowSlabs) {
        const int sl = blockIdx.z * kRowSlabs + threadIdx.x, lc = sl / v.H, h = sl - lc * v.H;
        s.in_pool[threadIdx.x] = ((long long)(2 * a.layer + lc) * v.P * v.H + h) * v.block;
        s.in_rows[threadIdx.x] = (((long long)lc * a.N + from) * v.H + h) * a.S * v.D;
    }
    if (threadIdx.x == 0)
        s.m = m;
    __syncthreads();
    return true;
}

// Calls f(token, part, slab) for all of a tile's parts (PARTS of a token) in all
// its slabs.  A thread has the same part in every slab, so that what it has to
// know of it is worked out once; where parts are few (a path's), threads are
// dealt out over slabs too.
template <typename F>
__device__ __forceinline__ void each_part(const Q4RowsArgs &a, const RowTile &s, int parts, F f)
{
    const int slabs = min(kRowSlabs, a.L * 2 * a.pool.H - (int)blockIdx.z * kRowSlabs), per = s.m * parts;
    const int rows = per < kRowThreads ? kRowThreads / per : 1;  // slabs at a time
    const int first = rows > 1 ? threadIdx.x / per : 0;
    if (first >= rows)
        return;
    for (int i = rows > 1 ? threadIdx.x - first * per : threadIdx.x; i < per; i += kRowThreads) {
        const int j = i / parts;
        if (s.at[j] >= 0)
            f(j, i - j * parts, first, rows, slabs);
        if (rows > 1)
            return;
    }
}

template <typename T>
__device__ __forceinline__ uint32_t top_bits();  // exponent of all ones
template <>
__device__ __forceinline__ uint32_t top_bits<__nv_bfloat16>() { return 0x7F80u; }
template <>
__device__ __forceinline__ uint32_t top_bits<__half>() { return 0x7C00u; }

template <typename T>
__device__ __forceinline__ float from_bits(uint32_t u)
{
    T x;
    const unsigned short h = (unsigned short)u;
    memcpy(&x, &h, 2);
    return (float)x;
}

// A thread takes a group, 64 bytes in, 16 bytes of codes and a scale out, and
// has the next slab's on their way meanwhile.  (Four threads a group read side by side,
// but each works out the scale: 32 prompts of 1050 tokens, 8 heads, 73 us against 33.)
template <typename T>
__global__ void __launch_bounds__(kRowThreads) store_q4_kernel(const Q4RowsArgs a)
{
    __shared__ RowTile s;
    if (!row_tile<true>(a, s))
        return;
    const int D = a.pool.D, groups = D / kGroup, codes = q4_codes(D) << a.pool.page_log2;  // of a block
    each_part(a, s, groups, [&](int j, int g, int first, int step, int slabs) {
        const T *src = static_cast<const T *>(a.src) + (long long)s.at[j] * D + g * kGroup;
        unsigned char *dst = a.pool.pool + s.page[j] * a.pool.page_bytes;
        const int code_at = s.in_page[j] * q4_codes(D) + g * 16, scale_at = codes + s.in_page[j] * groups + g;
        uint4 x[4], next[4];
        auto read = [&](int sl, uint4 *to) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                to[k] = __ldg(reinterpret_cast<const uint4 *>(src + s.in_rows[sl]) + k);
        };
        if (first < slabs)
            read(first, next);
#pragma unroll 1
        for (int sl = first; sl < slabs; sl += step) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[k] = next[k];
            if (sl + step < slabs)
                read(sl + step, next);
            const uint32_t *u = reinterpret_cast<const uint32_t *>(x);
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                top = __vmaxu2(top, u[k] & 0x7FFF7FFFu);
            top = max(top & 0xFFFFu, top >> 16);
            uint4 c = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
            int byte = kNanScale;
            if (top < top_bits<T>()) {
                const float amax = from_bits<T>(top);
                byte = q4_scale_byte(amax);
                const float sc = q4_scale(byte), r = q4_reciprocal(sc);
                const bool cut = amax > 7.4f * sc;  // the smallest and the largest scale may be too small for their group
                uint32_t *cw = reinterpret_cast<uint32_t *>(&c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = q4_level(from_bits<T>(u[4 * k + e / 2] >> (16 * (e & 1))), r);
                    if (cut)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[e] = fminf(fmaxf(y[e], -7.0f), 7.0f);
                    cw[k] = __byte_perm(q4_pack4(y[0], y[1], y[2], y[3]), q4_pack4(y[4], y[5], y[6], y[7]), 0x5410);
                }
            }
            unsigned char *blk = dst + s.in_pool[sl];
            *reinterpret_cast<uint4 *>(blk + code_at) = c;
            blk[scale_at] = (unsigned char)byte;
        }
    });
}

// Eight codes and their scale's byte -> eight values, in order.
template <typename T>
__device__ __forceinline__ uint4 q4_values(uint32_t word, uint32_t byte);
template <>
__device__ __forceinline__ uint4 q4_values<__nv_bfloat16>(uint32_t word, uint32_t byte)
{
    uint32_t x[4];
    q4_expand(word, Scale2Bf16(byte), x);
    return in_order(x);
}
template <>
__device__ __forceinline__ uint4 q4_values<__half>(uint32_t word, uint32_t byte)
{
    // in fp16's own units: 1024 + c less 1032, times s, both exact
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t y;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(and_or(word >> (4 * i), 0x000F000Fu, 0x64006400u)), "r"(0xE408E408u));
        x[i] = hmul2_bits(y, byte * 0x00800080u);
    }
    return in_order(x);
}

// A thread takes eight values: four bytes of codes in, 16 bytes out.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) load_q4_kernel(const Q4RowsArgs a)
{
    __shared__ RowTile s;
    if (!row_tile<false>(a, s))
        return;
    const int D = a.pool.D, groups = D / kGroup, codes = q4_codes(D) << a.pool.page_log2;
    constexpr int kAhead = 4;  // slabs whose loads are on their way at once
    each_part(a, s, D / 8, [&](int j, int p, int first, int step, int slabs) {
        T *dst = static_cast<T *>(a.dst) + (long long)s.at[j] * D + p * 8;
        const unsigned char *src = a.pool.pool + s.page[j] * a.pool.page_bytes;
        const int code_at = s.in_page[j] * q4_codes(D) + p * 4, scale_at = codes + s.in_page[j] * groups + p / 4;
        for (int sl = first; sl < slabs; sl += kAhead * step) {
            uint32_t word[kAhead], byte[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (sl + k * step < slabs) {
                    const unsigned char *blk = src + s.in_pool[sl + k * step];
                    word[k] = __ldg(reinterpret_cast<const uint32_t *>(blk + code_at));
                    byte[k] = __ldg(blk + scale_at);
                }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (sl + k * step < slabs)
                    *reinterpret_cast<uint4 *>(dst + s.in_rows[sl + k * step]) = q4_values<T>(word[k], byte[k]);
        }
    });
}

namespace {
dim3 rows_grid(const Q4RowsArgs &a)
{
    return dim3((unsigned)((a.T + kRowTokens - 1) / kRowTokens), (unsigned)a.B,
                (unsigned)((a.L * 2 * a.pool.H + kRowSlabs - 1) / kRowSlabs));
}
}  // namespace

cudaError_t launch_store_q4(const Q4RowsArgs &a, spec_dtype dt, cudaStream_t st)
{
    if (dt == SPEC_BF16)
        store_q4_kernel<__nv_bfloat16><<<rows_grid(a), kRowThreads, 0, st>>>(a);
    else
        store_q4_kernel<__half><<<rows_grid(a), kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_load_q4(const Q4RowsArgs &a, spec_dtype dt, cudaStream_t st)
{
    if (dt == SPEC_BF16)
        load_q4_kernel<__nv_bfloat16><<<rows_grid(a), kRowThreads, 0, st>>>(a);
    else
        load_q4_kernel<__half><<<rows_grid(a), kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace spec
