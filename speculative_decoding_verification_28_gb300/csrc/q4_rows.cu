// q4_rows.cu -- rows of 16-bit keys and values stored into pages of 4-bit codes,
// and loaded back.
//
// Each group of 32 values is read once and written once: 2 D + 17 D / 32 bytes a
// row, so HBM bounds both; a thread's group needs no other thread.  The
// products and quotients are exact (q4.cuh), so any order gives the same bytes.
#include "paged.h"
#include "q4.cuh"

namespace spec {

constexpr int kRowThreads = 128;
constexpr int kRowTokens = 64;  // tokens of a CTA
constexpr int kRowSlabs = 8;    // (layer, K or V, head) slabs of a CTA

// What a CTA knows of its sequence's tokens t0 .. t0 + m - 1.
struct RowTile {
    int m;
    int row;                   // row of the 16-bit block
    int at[kRowTokens];        // row within a slab of it, or -1: left out
    int page[kRowTokens];
    short in_page[kRowTokens];
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
    if (threadIdx.x == 0) {
        s.m = m;
        s.row = from;
    }
    __syncthreads();
    return true;
}

// block of a page's head in a slab of the pool; slab = (layer of the 16-bit block, K or V, head)
__device__ __forceinline__ unsigned char *block_of(const Q4RowsArgs &a, int lc, int h, int page)
{
    return a.pool.pool + ((((long long)(2 * a.layer + lc)) * a.pool.P + page) * a.pool.H + h) * a.pool.block;
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

// A thread takes a group: 64 bytes in, 16 bytes of codes and a scale out.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) store_q4_kernel(const Q4RowsArgs a)
{
    __shared__ RowTile s;
    if (!row_tile<true>(a, s))
        return;
    const int D = a.pool.D, H = a.pool.H, groups = D / kGroup, per_slab = s.m * groups;
    const int slab0 = blockIdx.z * kRowSlabs, slabs = min(kRowSlabs, a.L * 2 * H - slab0);
    const int codes = q4_codes(D) << a.pool.page_log2;  // of a block
    for (int w = threadIdx.x; w < slabs * per_slab; w += kRowThreads) {
        const int sl = w / per_slab, i = w - sl * per_slab, j = i / groups, g = i - j * groups;
        if (s.at[j] < 0)
            continue;
        const int lc = (slab0 + sl) / H, h = (slab0 + sl) - lc * H;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            static_cast<const T *>(a.src) + ((((long long)lc * a.N + s.row) * H + h) * a.S + s.at[j]) * D + g * kGroup);
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = __ldg(src + k);
        const uint32_t *u = reinterpret_cast<const uint32_t *>(x);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            top = __vmaxu2(top, u[k] & 0x7FFF7FFFu);
        top = max(top & 0xFFFFu, top >> 16);
        uint4 c = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        int byte = kNanScale;
        if (top < top_bits<T>()) {
            byte = q4_scale_byte(from_bits<T>(top));
            const float sc = q4_scale(byte), r = __frcp_rn(sc);
            uint32_t *cw = reinterpret_cast<uint32_t *>(&c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t word = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    word |= q4_code(from_bits<T>(u[4 * k + e / 2] >> (16 * (e & 1))), sc, r) << (4 * e);
                cw[k] = word;
            }
        }
        unsigned char *blk = block_of(a, lc, h, s.page[j]);
        *reinterpret_cast<uint4 *>(blk + s.in_page[j] * q4_codes(D) + g * 16) = c;
        blk[codes + s.in_page[j] * groups + g] = (unsigned char)byte;
    }
}

// A thread takes eight values: four bytes of codes in, 16 bytes out.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) load_q4_kernel(const Q4RowsArgs a)
{
    __shared__ RowTile s;
    if (!row_tile<false>(a, s))
        return;
    const int D = a.pool.D, H = a.pool.H, parts = D / 8, per_slab = s.m * parts;
    const int slab0 = blockIdx.z * kRowSlabs, slabs = min(kRowSlabs, a.L * 2 * H - slab0);
    const int codes = q4_codes(D) << a.pool.page_log2;
    for (int w = threadIdx.x; w < slabs * per_slab; w += kRowThreads) {
        const int sl = w / per_slab, i = w - sl * per_slab, j = i / parts, p = i - j * parts;
        if (s.at[j] < 0)
            continue;
        const int lc = (slab0 + sl) / H, h = (slab0 + sl) - lc * H;
        const unsigned char *blk = block_of(a, lc, h, s.page[j]);
        const uint32_t word = *reinterpret_cast<const uint32_t *>(blk + s.in_page[j] * q4_codes(D) + p * 4);
        const float sc = q4_scale(blk[codes + s.in_page[j] * (D / kGroup) + p / 4]);
        T y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = T((float)((int)(word >> (4 * e) & 15u) - 8) * sc);
        uint4 out;
        memcpy(&out, y, 16);
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.dst) + ((((long long)lc * a.N + s.row) * H + h) * a.S + s.at[j]) * D +
                                   p * 8) = out;
    }
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
