// attend_simt.cu -- attention on the CUDA cores: every storage type, any head
// size up to SPEC_MAX_HEAD_DIM and any alignment, in fp32 throughout.  It is
// the form for fp32 caches (the tensor cores have no fp32 product) and for
// head sizes the tensor-core kernel (attend_tc.cu) has no tile for.
//
//   o_r = sum_j e^(s_rj - m_r) v_j / sum_j e^(s_rj - m_r),  s_rj = scale q_r.k_j
//
// over the keys row r sees, in one pass with a running maximum m and sum.
// A unit has 16 query rows, a tile 64 keys: K and V tiles are brought to
// shared memory as fp32 once for the 16 rows; a thread forms 2 x 4 scores and
// 4 rows x 4 columns of the output.  Bound by the FMA pipe from about 20 rows
// a key head on, by HBM below.
#include "attend_common.cuh"

namespace spec {

constexpr int kSimtThreads = 128;
constexpr int kSimtRows = 16;
constexpr int kSimtKeys = 64;

// shared memory, in floats: q[16][DP], k[64][DP + 4], v[64][DP], p[64][16];
// DP = D rounded up to 4 (the +4 spreads a column of keys over the banks)
__host__ __device__ inline int simt_dp(int D) { return (D + 3) & ~3; }
inline size_t simt_smem(int D)
{
    const int dp = simt_dp(D);
    return sizeof(float) * ((size_t)kSimtRows * dp + (size_t)kSimtKeys * (dp + 4) + (size_t)kSimtKeys * dp +
                            kSimtKeys * kSimtRows);
}

// rows x D elements at src (row step `step`) to fp32 rows of `ld` floats;
// rows from `have` on and columns from D on are zero
template <typename T>
__device__ __forceinline__ void load_rows(const T *src, long long step, int have, int rows, int D, float *dst, int ld)
{
    const int dp = simt_dp(D), quads = dp / 4;
    const bool vec = D % 4 == 0 && (reinterpret_cast<uintptr_t>(src) % (4 * sizeof(T))) == 0;
    for (int w = threadIdx.x; w < rows * quads; w += kSimtThreads) {
        const int r = w / quads, c = (w - r * quads) * 4;
        float4 f = make_float4(0, 0, 0, 0);
        if (r < have) {
            const T *s = src + r * step + c;
            if (vec) {
                if constexpr (sizeof(T) == 4) {
                    f = __ldg(reinterpret_cast<const float4 *>(s));
                } else {
                    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(s));
                    float x[8];
                    Storage<T>::unpack(make_uint4(u.x, u.y, 0, 0), x);
                    f = make_float4(x[0], x[1], x[2], x[3]);
                }
            } else {
                f.x = Storage<T>::at(s, 0);
                f.y = c + 1 < D ? Storage<T>::at(s, 1) : 0.0f;
                f.z = c + 2 < D ? Storage<T>::at(s, 2) : 0.0f;
                f.w = c + 3 < D ? Storage<T>::at(s, 3) : 0.0f;
            }
        }
        *reinterpret_cast<float4 *>(dst + (size_t)r * ld + c) = f;
    }
}

// CB: column blocks of 128 of the output (1: D <= 128, 2: D <= 256)
template <typename T, int CB, bool PROMPT>
__global__ void __launch_bounds__(kSimtThreads) attend_simt_kernel(AttendArgs a)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ uint32_t s_scan[kSimtThreads / 32];
    __shared__ Run s_run;
    __shared__ float s_f[kSimtRows], s_m[kSimtRows], s_l[kSimtRows];
    __shared__ int s_last;
    const int D = a.cache.D, dp = simt_dp(D);
    float *q = smem, *k = q + kSimtRows * dp, *v = k + kSimtKeys * (dp + 4), *p = v + kSimtKeys * dp;
    const Shape sh{kSimtKeys, kSimtRows, a.G};
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;

    AttendUnit u;
    bool have;
    if constexpr (PROMPT) {
        have = prompt_unit(a, sh, u);
    } else {
        if (t == 0)
            s_run.begin = s_run.end = 0;
        find_run<kSimtThreads>(a, sh, s_scan, &s_run);
        __syncthreads();
    }
    UnitWalk walk(a, sh, PROMPT ? Run{} : s_run);
    if constexpr (!PROMPT)
        have = walk.next(u);
    const long long slab = (long long)a.cache.S * D;
    while (have) {
        const T *kc = reinterpret_cast<const T *>(a.cache.kv) +
                      (a.cache.k_slab + (long long)u.seq.row * a.cache.H + u.h) * slab + (long long)u.seq.slot0 * D;
        const T *vc = kc + (a.cache.v_slab - a.cache.k_slab) * slab;
        // query rows: row r at row_place
        for (int w = t; w < kSimtRows * dp; w += kSimtThreads) {
            const int r = w / dp, c = w - r * dp;
            q[w] = r < u.n_rows && c < D
                       ? Storage<T>::at(reinterpret_cast<const T *>(a.q) + row_place(a, u, r), c) * a.scale_log2
                       : 0.0f;
        }
        if (t < kSimtRows) {
            s_m[t] = -INFINITY;
            s_l[t] = 0.0f;
        }
        float acc[CB][4][4] = {};
        const int rg = warp * 4;  // rows rg .. rg + 3 of the output and of the softmax
        __syncthreads();
        for (int tile = u.tile; tile < u.tile_end; ++tile) {
            const bool nodes = !PROMPT && tile == u.n_tiles - 1;
            int keys;  // real keys of the tile; the rest of it is zero
            const T *ks, *vs;
            if (nodes) {
                keys = u.seq.n;
                if (a.seq.staged) {
                    const long long at = ((long long)u.b * a.cache.H + u.h) * a.seq.T * D, sl = (long long)a.seq.T * D;
                    ks = reinterpret_cast<const T *>(a.staged) + a.st_k * sl + at;
                    vs = reinterpret_cast<const T *>(a.staged) + a.st_v * sl + at;
                } else {
                    ks = kc + (long long)u.seq.prefix * D;
                    vs = vc + (long long)u.seq.prefix * D;
                }
            } else {
                const int k0 = tile * kSimtKeys;
                const int end = PROMPT ? u.seen_last : u.seq.prefix;
                keys = min(kSimtKeys, end - k0);
                ks = kc + (long long)k0 * D;
                vs = vc + (long long)k0 * D;
            }
            load_rows<T>(ks, D, keys, kSimtKeys, D, k, dp + 4);
            load_rows<T>(vs, D, keys, kSimtKeys, D, v, dp);
            __syncthreads();
            // scores: rows 2 (t / 16) + {0, 1}, keys t % 16 + {0, 16, 32, 48}
            {
                float s[2][4] = {};
                const int r0 = (t >> 4) * 2, kk = t & 15;
                for (int c = 0; c < dp; c += 4) {
                    const float4 q0 = *reinterpret_cast<const float4 *>(q + r0 * dp + c);
                    const float4 q1 = *reinterpret_cast<const float4 *>(q + (r0 + 1) * dp + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 x = *reinterpret_cast<const float4 *>(k + (kk + 16 * j) * (dp + 4) + c);
                        s[0][j] = fmaf(q0.x, x.x, fmaf(q0.y, x.y, fmaf(q0.z, x.z, fmaf(q0.w, x.w, s[0][j]))));
                        s[1][j] = fmaf(q1.x, x.x, fmaf(q1.y, x.y, fmaf(q1.z, x.z, fmaf(q1.w, x.w, s[1][j]))));
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = (u.row0 + r0 + i) / a.G;
                    int lim = keys;  // keys of this tile the row sees, as a count ...
                    uint64_t bits = ~0ull;  // ... or as a mask
                    if (PROMPT)
                        lim = min(keys, u.seq.prefix + tok + 1 - tile * kSimtKeys);
                    else if (nodes) {
                        if (r0 + i < u.n_rows)
                            bits = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok] : (2ull << tok) - 1;
                        else
                            bits = 0;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = kk + 16 * j;
                        p[key * kSimtRows + r0 + i] = key < lim && (bits >> key & 1) ? s[i][j] : -INFINITY;
                    }
                }
            }
            __syncthreads();
            // softmax: warp w has rows 4 w .. 4 w + 3, lane l keys l and l + 32
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = rg + i;
                const float x0 = p[lane * kSimtRows + r], x1 = p[(lane + 32) * kSimtRows + r];
                float mx = fmaxf(x0, x1);
#pragma unroll
                for (int m = 16; m > 0; m >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, m));
                const float m_old = s_m[r], m_new = fmaxf(m_old, mx);
                const float m0 = m_new == -INFINITY ? 0.0f : m_new;  // nothing seen yet: every weight is 0
                // a place that is not seen has weight 0, whatever its score
                const float e0 = exp2f(x0 - m0), e1 = exp2f(x1 - m0);
                p[lane * kSimtRows + r] = e0;
                p[(lane + 32) * kSimtRows + r] = e1;
                float sum = e0 + e1;
#pragma unroll
                for (int m = 16; m > 0; m >>= 1)
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
                __syncwarp();
                if (lane == 0) {
                    const float f = exp2f(m_old - m0);
                    s_f[r] = f;
                    s_l[r] = fmaf(s_l[r], f, sum);
                    s_m[r] = m_new;
                }
            }
            __syncwarp();
            // output: the same rows, columns 4 lane + 128 cb ..; a weight of 0
            // takes nothing, so a value that is not finite stays with the rows
            // that see it
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = s_f[rg + i];
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[cb][i][e] *= f[i];
            for (int key = 0; key < keys; ++key) {
                const float4 w = *reinterpret_cast<const float4 *>(p + key * kSimtRows + rg);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    const int c = 4 * lane + 128 * cb;
                    if (c < dp) {
                        const float4 x = *reinterpret_cast<const float4 *>(v + (size_t)key * dp + c);
                        const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (ww[i] != 0.0f) {
                                acc[cb][i][0] = fmaf(ww[i], x.x, acc[cb][i][0]);
                                acc[cb][i][1] = fmaf(ww[i], x.y, acc[cb][i][1]);
                                acc[cb][i][2] = fmaf(ww[i], x.z, acc[cb][i][2]);
                                acc[cb][i][3] = fmaf(ww[i], x.w, acc[cb][i][3]);
                            }
                        }
                    }
                }
            }
            __syncthreads();
        }
        const bool whole = u.n_parts == 1;
        float *slot = whole ? nullptr : part_slot<kSimtRows>(a, blockIdx.x, u.part);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rg + i;
            if (r >= u.n_rows)
                continue;
            const float l = s_l[r], inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 4 * lane + 128 * cb + e;
                    if (c < D) {
                        if (whole)
                            reinterpret_cast<T *>(a.out)[row_place(a, u, r) + c] = round_to<T>(acc[cb][i][e] * inv);
                        else
                            __stcg(slot + (size_t)r * dp + c, acc[cb][i][e]);
                    }
                }
            if (!whole && lane == 0) {
                __stcg(slot + (size_t)kSimtRows * dp + r, s_m[r]);
                __stcg(slot + (size_t)kSimtRows * dp + kSimtRows + r, l);
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (t == 0) {
                int *cnt = part_counter(a, u.first_cta);
                s_last = atomicAdd(cnt, 1) == u.n_parts - 1;
                if (s_last)
                    *cnt = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_parts<T, kSimtRows>(a, u, warp, kSimtThreads / 32);
            }
        }
        __syncthreads();  // q, s_l and s_last are rewritten next
        if constexpr (PROMPT)
            have = false;
        else
            have = walk.next(u);
    }
}

template <typename T, int CB, bool PROMPT>
cudaError_t launch_simt(const AttendArgs &a, cudaStream_t st)
{
    const size_t smem = simt_smem(a.cache.D);
    cudaError_t e = cudaFuncSetAttribute(attend_simt_kernel<T, CB, PROMPT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess)
        return e;
    dim3 grid(kAttendCtas);
    if (PROMPT) {
        const long long units = ((long long)a.seq.M * a.G + kSimtRows - 1) / kSimtRows + a.seq.B;
        grid = dim3((unsigned)units, (unsigned)a.cache.H);
    }
    attend_simt_kernel<T, CB, PROMPT><<<grid, kSimtThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt_t(const AttendArgs &a, cudaStream_t st)
{
    if (a.cache.D <= 128)
        return a.seq.cu ? launch_simt<T, 1, true>(a, st) : launch_simt<T, 1, false>(a, st);
    return a.seq.cu ? launch_simt<T, 2, true>(a, st) : launch_simt<T, 2, false>(a, st);
}

size_t attend_workspace(int T, int Hq, int H, int D)
{
    const size_t simt = align256(kPartHead + 2 * kAttendCtas * part_floats<kSimtRows>(D) * sizeof(float));
    const size_t tc = D == 64 || D == 128 ? attend_tc_workspace(T, Hq, H, D) : 0;
    return simt > tc ? simt : tc;
}

cudaError_t launch_attend(const AttendArgs &a, spec_dtype dt, cudaStream_t st)
{
    if (attend_tc_takes(a, dt))
        return launch_attend_tc(a, dt, st);
    switch (dt) {
    case SPEC_F32:
        return launch_simt_t<float>(a, st);
    case SPEC_BF16:
        return launch_simt_t<__nv_bfloat16>(a, st);
    default:
        return launch_simt_t<__half>(a, st);
    }
}

}  // namespace spec
