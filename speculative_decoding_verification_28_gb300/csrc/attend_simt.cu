// attend_simt.cu -- attention on the CUDA cores: every storage type, any head
// size up to SPEC_MAX_HEAD_DIM and any alignment, in fp32 throughout.  It is
// the form for fp32 caches (the tensor cores have no fp32 product) and for
// head sizes the tensor-core kernels have no tile for.
//
//   o_r = sum_j e^(s_rj - m_r) v_j / sum_j e^(s_rj - m_r),  s_rj = scale q_r.k_j
//
// over the keys row r sees, in one pass with a running maximum m and sum.
// A unit has 16 IR query rows, a tile 64 keys.  256 threads stand in 16 x 16:
// thread (ty, tx) forms the scores of rows IR ty .. and keys tx + 16 j, and
// the output of the same rows and columns 4 tx + 64 j, so that a row's maximum,
// sum and rescaling stay with the 16 lanes of its ty.  K and then V take the
// same shared buffer as fp32, the next of them on its way in registers; the
// weights pass through shared memory.  IR = 4 has 64 FMAs to 8 shared loads in
// the scores, 32 to 3 in the output; IR = 1, for up to 16 rows, is bound by shared
// memory and latency (4 rows, 32 sequences: 162 us, 365 with IR = 4; 16 rows, 16
// sequences: 176, 391).  fp32 prompts (2 of 2048 tokens, 32 / 8 heads of 128)
// run at 29 TFLOP/s, 32 rounds of 64 nodes and 28 / 4 heads at 25: the FMA pipes
// are 40% busy, shared memory 60%, issue slots 61%, and what is waited for are
// shared loads, with 16 warps an SM (two CTAs of 128 registers a thread; spills
// are 0.5% of the instructions).  The smallest rounds take 9 us, all latency.
#include "attend_common.cuh"
#include "verify_common.cuh"

namespace spec {

constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 64;
constexpr int kSimtCtas = 2 * kAttendCtas;

__host__ __device__ inline int simt_dp(int D) { return (D + 3) & ~3; }
// q[rows][dp], k or v[64][dp + 4], p[64][rows + 4], in floats (the + 4 spread
// columns over the banks)
inline size_t simt_smem(int D, int rows)
{
    const size_t dp = simt_dp(D);
    return sizeof(float) * (rows * dp + kSimtKeys * (dp + 4) + kSimtKeys * (size_t)(rows + 4));
}

// four elements from p on as fp32; those from `left` on are zero
template <typename T>
__device__ __forceinline__ float4 load4(const T *p, int left, bool vec)
{
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            return __ldg(reinterpret_cast<const float4 *>(p));
        } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
            float x[8];
            Storage<T>::unpack(make_uint4(u.x, u.y, 0, 0), x);
            return make_float4(x[0], x[1], x[2], x[3]);
        }
    }
    float4 f;
    f.x = Storage<T>::at(p, 0);
    f.y = left > 1 ? Storage<T>::at(p, 1) : 0.0f;
    f.z = left > 2 ? Storage<T>::at(p, 2) : 0.0f;
    f.w = left > 3 ? Storage<T>::at(p, 3) : 0.0f;
    return f;
}

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

// maximum / sum over the 16 lanes of a ty
__device__ __forceinline__ float max16(float x)
{
#pragma unroll
    for (int m = 8; m > 0; m >>= 1)
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, m));
    return x;
}
__device__ __forceinline__ float sum16(float x)
{
#pragma unroll
    for (int m = 8; m > 0; m >>= 1)
        x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
    return x;
}

// CB: blocks of 64 columns (D <= 64 CB)
template <typename T, int IR, int CB, bool PROMPT>
__global__ void __launch_bounds__(kSimtThreads, CB <= 2 ? 2 : 1) attend_simt_kernel(AttendArgs a)
{
    constexpr int ROWS = 16 * IR;
    extern __shared__ __align__(16) float smem[];
    __shared__ uint32_t s_scan[kSimtThreads / 32];
    __shared__ Run s_run;
    __shared__ int s_last;
    const int D = a.cache.D, dp = simt_dp(D), ld = dp + 4;
    float *q = smem, *kv = q + ROWS * dp, *p = kv + kSimtKeys * ld;
    const Shape sh{kSimtKeys, ROWS, a.G};
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;

    AttendUnit u;
    bool have;
    if constexpr (PROMPT) {
        have = prompt_unit(a, sh, u);
    } else {
        if (t == 0)
            s_run.begin = s_run.end = 0;
        __syncthreads();
        find_run<kSimtThreads>(a, sh, s_scan, &s_run);
        __syncthreads();
    }
    UnitWalk<> walk(a, sh, PROMPT ? Run{} : s_run);
    if constexpr (!PROMPT)
        have = walk.next(u);
    const long long slab = (long long)a.cache.S * D;
    while (have) {
        const T *kc = reinterpret_cast<const T *>(a.cache.kv) +
                      (a.cache.k_slab + (long long)u.seq.row * a.cache.H + u.h) * slab + (long long)u.seq.slot0 * D;
        const T *vc = kc + (a.cache.v_slab - a.cache.k_slab) * slab;
        // K or V of a tile: where its keys are, how many are real
        struct Src {
            const T *at;
            int keys;
            bool nodes;
        };
        auto tile_src = [&](int tile, bool v) -> Src {
            Src s;
            s.nodes = !PROMPT && tile == u.n_tiles - 1;
            s.at = v ? vc : kc;
            if (s.nodes) {
                s.keys = u.seq.n;
                if (a.seq.staged)
                    s.at = reinterpret_cast<const T *>(a.staged) +
                           ((v ? a.st_v : a.st_k) + (long long)u.b * a.cache.H + u.h) * a.seq.T * D;
                else
                    s.at += (long long)u.seq.prefix * D;
            } else {
                s.keys = min(kSimtKeys, (PROMPT ? u.seen_last : u.seq.prefix) - tile * kSimtKeys);
                s.at += (long long)tile * kSimtKeys * D;
            }
            return s;
        };
        // this thread's part of a tile: rows ty + 16 j, quads tx + 16 b
        float4 pre[4 * CB];
        auto fetch = [&](const Src &s) {
            const bool vec = D % 4 == 0 && reinterpret_cast<uintptr_t>(s.at) % (4 * sizeof(T)) == 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int b = 0; b < CB; ++b) {
                    const int r = ty + 16 * j, c = 4 * (tx + 16 * b);
                    pre[j * CB + b] = r < s.keys && c < D ? load4<T>(s.at + (long long)r * D + c, D - c, vec)
                                                          : make_float4(0, 0, 0, 0);
                }
        };
        auto put = [&]() {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int b = 0; b < CB; ++b) {
                    const int c = 4 * (tx + 16 * b);
                    if (c < dp)
                        *reinterpret_cast<float4 *>(kv + (ty + 16 * j) * ld + c) = pre[j * CB + b];
                }
        };
        fetch(tile_src(u.tile, false));
        // query rows, scaled
        for (int r = ty; r < ROWS; r += 16) {
            const T *src = reinterpret_cast<const T *>(a.q) + (r < u.n_rows ? row_place(a, u, r) : 0);
            for (int c = tx; c < dp; c += 16)
                q[r * dp + c] = r < u.n_rows && c < D ? Storage<T>::at(src, c) * a.scale_log2 : 0.0f;
        }
        float m[IR], l[IR], acc[IR][4 * CB];
        uint64_t bits[IR];  // nodes that the row sees
        int tok[IR];
#pragma unroll
        for (int i = 0; i < IR; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 4 * CB; ++e)
                acc[i][e] = 0.0f;
            const int r = IR * ty + i;
            tok[i] = (u.row0 + r) / a.G;
            bits[i] = 0;
            if (!PROMPT && r < u.n_rows && u.tile_end == u.n_tiles)
                bits[i] = a.mask ? a.mask[(size_t)u.b * a.seq.T + tok[i]] : (2ull << tok[i]) - 1;
        }
        put();
        __syncthreads();
        for (int tile = u.tile; tile < u.tile_end; ++tile) {
            const Src vs = tile_src(tile, true);
            fetch(vs);  // V, while the scores form
            float s[IR][4];
#pragma unroll
            for (int i = 0; i < IR; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[i][j] = 0.0f;
#pragma unroll 4
            for (int c = 0; c < dp; c += 4) {
                float4 x[IR], y[4];
#pragma unroll
                for (int i = 0; i < IR; ++i)
                    x[i] = *reinterpret_cast<const float4 *>(q + (IR * ty + i) * dp + c);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[j] = *reinterpret_cast<const float4 *>(kv + (tx + 16 * j) * ld + c);
#pragma unroll
                for (int i = 0; i < IR; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(x[i].x, y[j].x,
                                       fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
            }
            // places the row does not see
            bool hidden = vs.nodes || vs.keys < kSimtKeys;
#pragma unroll
            for (int i = 0; i < IR; ++i) {
                int lim = vs.keys;
                if (PROMPT)
                    lim = min(lim, u.seq.prefix + tok[i] + 1 - tile * kSimtKeys);
                hidden |= lim < kSimtKeys;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = tx + 16 * j;
                    if (key >= lim || (vs.nodes && !(bits[i] >> key & 1)))
                        s[i][j] = -INFINITY;
                }
            }
            float w[4][IR];
#pragma unroll
            for (int i = 0; i < IR; ++i) {
                const float mx = fmaxf(m[i], max16(fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]))));
                const float m0 = mx == -INFINITY ? 0.0f : mx;  // nothing seen yet: every weight is 0
                const float f = exp2f(m[i] - m0);
                m[i] = mx;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j][i] = exp2f(s[i][j] - m0);
                    sum += w[j][i];
                }
                l[i] = fmaf(l[i], f, sum16(sum));
#pragma unroll
                for (int e = 0; e < 4 * CB; ++e)
                    acc[i][e] *= f;
            }
            __syncthreads();  // K has been read
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float *dst = p + (tx + 16 * j) * (ROWS + 4) + IR * ty;
                if constexpr (IR == 4)
                    *reinterpret_cast<float4 *>(dst) = make_float4(w[j][0], w[j][1], w[j][2], w[j][3]);
                else
                    dst[0] = w[j][0];
            }
            put();
            if (tile + 1 < u.tile_end)
                fetch(tile_src(tile + 1, false));  // the next K, while the output forms
            const bool any_hidden = __syncthreads_or(hidden);
            auto product = [&](auto guarded) {
#pragma unroll 4
                for (int key = 0; key < vs.keys; ++key) {
                    float ww[IR];
                    if constexpr (IR == 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(p + key * (ROWS + 4) + 4 * ty);
                        ww[0] = x.x;
                        ww[1] = x.y;
                        ww[2] = x.z;
                        ww[3] = x.w;
                    } else {
                        ww[0] = p[key * (ROWS + 4) + ty];
                    }
#pragma unroll
                    for (int b = 0; b < CB; ++b) {
                        const int c = 4 * (tx + 16 * b);
                        if (CB * 64 > dp && c >= dp)
                            continue;
                        const float4 x = *reinterpret_cast<const float4 *>(kv + key * ld + c);
#pragma unroll
                        for (int i = 0; i < IR; ++i) {
                            // a weight of 0 takes nothing where some rows do not
                            // see the key: its value may be anything
                            if (!decltype(guarded)::value || ww[i] != 0.0f) {
                                acc[i][4 * b] = fmaf(ww[i], x.x, acc[i][4 * b]);
                                acc[i][4 * b + 1] = fmaf(ww[i], x.y, acc[i][4 * b + 1]);
                                acc[i][4 * b + 2] = fmaf(ww[i], x.z, acc[i][4 * b + 2]);
                                acc[i][4 * b + 3] = fmaf(ww[i], x.w, acc[i][4 * b + 3]);
                            }
                        }
                    }
                }
            };
            if (any_hidden)
                product(Flag<true>{});
            else
                product(Flag<false>{});
            __syncthreads();  // V and the weights have been read
            if (tile + 1 < u.tile_end) {
                put();
                __syncthreads();
            }
        }
        const bool whole = u.n_parts == 1;
        float *slot = whole ? nullptr : part_slot<ROWS>(a, blockIdx.x, u.part);
#pragma unroll
        for (int i = 0; i < IR; ++i) {
            const int r = IR * ty + i;
            if (r >= u.n_rows)
                continue;
            const float f = !whole ? 1.0f : l[i] > 0.0f || l[i] != l[i] ? 1.0f / l[i] : 0.0f;
            T *dst = reinterpret_cast<T *>(a.out) + row_place(a, u, r);
#pragma unroll
            for (int b = 0; b < CB; ++b) {
                const int c = 4 * (tx + 16 * b);
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < D)
                            dst[c + e] = round_to<T>(acc[i][4 * b + e] * f);
                } else if (c < dp) {
                    __stcg(reinterpret_cast<float4 *>(slot + part_quad<ROWS>(c / 4, r)),
                           make_float4(acc[i][4 * b], acc[i][4 * b + 1], acc[i][4 * b + 2], acc[i][4 * b + 3]));
                }
            }
            if (!whole && tx == 0) {
                __stcg(slot + (size_t)ROWS * dp + r, m[i]);
                __stcg(slot + (size_t)ROWS * dp + ROWS + r, l[i]);
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
                join_parts<T, ROWS>(a, u, t, kSimtThreads, [] {
                    __threadfence();
                    __syncthreads();
                    return true;
                });
            }
        }
        __syncthreads();  // q, kv and s_last are rewritten next
        if constexpr (PROMPT)
            have = false;
        else
            have = walk.next(u);
    }
}

template <typename T, int IR, int CB, bool PROMPT>
cudaError_t launch_simt(const AttendArgs &a, cudaStream_t st)
{
    constexpr int ROWS = 16 * IR;
    const size_t smem = simt_smem(a.cache.D, ROWS);
    cudaError_t e = cudaFuncSetAttribute(attend_simt_kernel<T, IR, CB, PROMPT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    dim3 grid(kSimtCtas);
    if (PROMPT) {
        const long long units = (long long)a.seq.M * a.G / ROWS + a.seq.B;
        grid = dim3((unsigned)units, (unsigned)a.cache.H);
    }
    attend_simt_kernel<T, IR, CB, PROMPT><<<grid, kSimtThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int CB>
cudaError_t launch_simt_cb(const AttendArgs &a, cudaStream_t st)
{
    if (a.seq.cu)
        return launch_simt<T, 4, CB, true>(a, st);
    return a.seq.T * a.G <= 16 ? launch_simt<T, 1, CB, false>(a, st) : launch_simt<T, 4, CB, false>(a, st);
}

template <typename T>
cudaError_t launch_simt_t(const AttendArgs &a, cudaStream_t st)
{
    if (a.cache.D <= 64)
        return launch_simt_cb<T, 1>(a, st);
    return a.cache.D <= 128 ? launch_simt_cb<T, 2>(a, st) : launch_simt_cb<T, 4>(a, st);
}

size_t attend_workspace(int T, int Hq, int H, int D)
{
    const size_t simt = align256(kPartHead + 2 * kSimtCtas * part_floats<64>(D) * sizeof(float));
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
