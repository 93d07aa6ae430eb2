// tree.cu -- drafted trees: the masks and depths attention needs, greedy
// verification along the accepted path, and the commit of that path's staged
// keys and values into the cache.
//
// A tree of n <= T <= 64 nodes: node 0 is the last committed token (the
// root), node i > 0 a proposal with parent[i] < i.  Row alignment as for a
// chain ("Chapter 10 Speculative Decoding (Code Walkthrough)", §3.3): the
// target's row of a node predicts the token after that node's path.
#include "forward.h"
#include "spec_common.cuh"
#include "verify_common.cuh"

namespace spec {

// ---------------------------------------------------------------------------
// masks and depths
// ---------------------------------------------------------------------------
// One warp per sequence; lane l keeps nodes l and l + 32.  A node's mask is
// its own bit and its parent's mask: each node walks up its parents (at most
// 63 shuffles, every lane in step).
__global__ void __launch_bounds__(32) tree_plan_kernel(int B, int T, const int32_t *parent, const int32_t *n_nodes,
                                                       uint64_t *mask, int32_t *depth, uint32_t *flags)
{
    const int b = blockIdx.x, lane = threadIdx.x;
    const int n = n_nodes ? n_nodes[b] : T;
    bool ok = n >= 0 && n <= T;
    int up[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int i = lane + 32 * s;
        up[s] = -1;
        if (ok && i < n) {
            up[s] = parent[(size_t)b * T + i];
            ok = ok && (i == 0 ? up[s] == -1 : (up[s] >= 0 && up[s] < i));
        }
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
    uint64_t m[2] = {0, 0};
    int d[2] = {0, 0}, at[2];
    at[0] = ok && lane < n ? lane : -1;
    at[1] = ok && lane + 32 < n ? lane + 32 : -1;
    while (__any_sync(0xFFFFFFFFu, at[0] >= 0 || at[1] >= 0)) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int i = at[s];
            if (i >= 0)
                m[s] |= 1ull << i;
            const int lo = __shfl_sync(0xFFFFFFFFu, up[0], i & 31), hi = __shfl_sync(0xFFFFFFFFu, up[1], i & 31);
            if (i >= 0) {
                at[s] = i < 32 ? lo : hi;
                d[s] += at[s] >= 0;
            }
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int i = lane + 32 * s;
        if (i < T) {
            mask[(size_t)b * T + i] = m[s];
            depth[(size_t)b * T + i] = d[s];
        }
    }
    if (lane == 0 && flags)
        flags[b] = ok ? 0u : SPEC_FLAG_BAD_TREE;
}

cudaError_t launch_tree_plan(int B, int T, const int32_t *parent, const int32_t *n_nodes, uint64_t *mask,
                             int32_t *depth, uint32_t *flags, cudaStream_t st)
{
    tree_plan_kernel<<<(unsigned)B, 32, 0, st>>>(B, T, parent, n_nodes, mask, depth, flags);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// greedy verification
// ---------------------------------------------------------------------------
constexpr int kTreeThreads = 256;

size_t tree_workspace(int B) { return align256((size_t)(B > 0 ? B : 0) * 8); }

// argmax key of a row: largest value, lowest index, NaN above all
template <typename T>
__device__ uint64_t row_key(const T *row, int lo, int hi)
{
    uint64_t key = 0;
    for (int i = lo + threadIdx.x; i < hi; i += kTreeThreads) {
        const uint64_t k = argmax_key(Storage<T>::at(row, i), (uint32_t)i);
        key = k > key ? k : key;
    }
    return key;
}

// One CTA walks one sequence: the row of the node it stands on, its argmax,
// the lowest child that proposed that token.
template <typename T>
__global__ void __launch_bounds__(kTreeThreads) verify_tree_kernel(TreeArgs a)
{
    __shared__ uint64_t s_red[kTreeThreads / 32];
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const int n = a.n_nodes ? a.n_nodes[b] : a.T;
    const int rem = a.remaining ? a.remaining[b] : 0x7FFFFFFF;
    bool ok = n >= 0 && n <= a.T;
    int up[2] = {-1, -1}, tok[2] = {-1, -1};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int i = lane + 32 * s;
        if (ok && i < n) {
            up[s] = a.parent[(size_t)b * a.T + i];
            tok[s] = a.tokens[(size_t)b * a.T + i];
            ok = ok && (i == 0 ? up[s] == -1 : (up[s] >= 0 && up[s] < i));
        }
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
    int emit = 0, accept = 0, at = 0;
    int out_t[2] = {-1, -1}, out_p[2] = {-1, -1};  // entry lane + 32 s
    bool live = ok && n > 0 && rem > 0;
    while (live) {
        const T *row = reinterpret_cast<const T *>(a.logits) + ((size_t)b * a.T + at) * a.V;
        const int t = (int)key_index(block_max_u64(row_key<T>(row, 0, a.V), s_red));
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (emit == lane + 32 * s) {
                out_t[s] = t;
                out_p[s] = at;
            }
        ++emit;
        const unsigned lo = __ballot_sync(0xFFFFFFFFu, up[0] == at && tok[0] == t);
        const unsigned hi = __ballot_sync(0xFFFFFFFFu, up[1] == at && tok[1] == t);
        const int child = lo ? __ffs(lo) - 1 : hi ? __ffs(hi) + 31 : -1;
        accept += child >= 0;
        live = child >= 0 && emit < rem && !(a.eos >= 0 && t == a.eos);
        at = child;
    }
    if (threadIdx.x < 32) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int i = lane + 32 * s;
            if (i < a.T) {
                a.out_tokens[(size_t)b * a.T + i] = out_t[s];
                a.path[(size_t)b * a.T + i] = out_p[s];
            }
        }
        if (lane == 0) {
            a.n_emit[b] = emit;
            a.n_accept[b] = accept;
            if (a.flags)
                a.flags[b] = ok ? 0u : SPEC_FLAG_BAD_TREE;
        }
    }
}

cudaError_t launch_verify_tree(const TreeArgs &a, spec_dtype dt, cudaStream_t st)
{
    switch (dt) {
    case SPEC_F32:
        verify_tree_kernel<float><<<(unsigned)a.B, kTreeThreads, 0, st>>>(a);
        break;
    case SPEC_BF16:
        verify_tree_kernel<__nv_bfloat16><<<(unsigned)a.B, kTreeThreads, 0, st>>>(a);
        break;
    default:
        verify_tree_kernel<__half><<<(unsigned)a.B, kTreeThreads, 0, st>>>(a);
        break;
    }
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
// Sequence b's staged rows path[b][0 .. n_emit) of every (layer, K/V, head)
// slab go to slots pad + len - 1 .. of the cache: 2 * n_emit * D * sizeof
// bytes a slab, HBM at best, a few MB and so a latency in practice.  One CTA
// per (sequence, kCommitSlabs slabs); a thread moves one E of a row.
constexpr int kCommitThreads = 128;
constexpr int kCommitSlabs = 8;

template <typename E>
__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(CommitArgs a)
{
    __shared__ int s_path[SPEC_MAX_NODES];
    const int b = blockIdx.y;
    const int n = a.n_emit[b], row = a.idx ? a.idx[b] : b;
    const long long slot = (a.pad ? a.pad[b] : 0) + (long long)a.len[b] - 1;
    bool ok = n >= 0 && n <= a.T && row >= 0 && row < a.N && a.len[b] >= 1 && (!a.pad || a.pad[b] >= 0) &&
              slot + n <= a.S;
    for (int j = threadIdx.x; j < a.T; j += kCommitThreads) {
        const int p = a.path[(size_t)b * a.T + j];
        s_path[j] = p;
        if (ok && j < n)
            ok = p >= 0 && p < a.T;
    }
    const bool twice = repeated_row(a.idx, a.B, row);
    ok = __syncthreads_and(ok && !twice);
    if (threadIdx.x == 0 && blockIdx.x == 0 && a.flags)
        a.flags[b] = ok ? 0u : SPEC_FLAG_BAD_STATE;
    if (!ok)
        return;
    const int per_row = (int)((long long)a.D * a.elt_bytes / (long long)sizeof(E));
    const int per_slab = n * per_row;
    const int slab0 = blockIdx.x * kCommitSlabs, slabs = min(kCommitSlabs, a.L * 2 * a.H - slab0);
    for (int w = threadIdx.x; w < slabs * per_slab; w += kCommitThreads) {
        const int s = slab0 + w / per_slab, r = w % per_slab;
        const int j = r / per_row, e = r % per_row;
        const int lc = s / a.H, h = s % a.H;
        const E *src = reinterpret_cast<const E *>(a.staged) +
                       ((((long long)lc * a.B + b) * a.H + h) * a.T + s_path[j]) * per_row + e;
        E *dst = reinterpret_cast<E *>(a.kv) + ((((long long)lc * a.N + row) * a.H + h) * a.S + slot + j) * per_row + e;
        *dst = *src;
    }
}

cudaError_t launch_commit_tree(const CommitArgs &a, cudaStream_t st)
{
    const dim3 grid((unsigned)((a.L * 2 * a.H + kCommitSlabs - 1) / kCommitSlabs), (unsigned)a.B);
    const long long row_bytes = (long long)a.D * a.elt_bytes;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.staged) | reinterpret_cast<uintptr_t>(a.kv);
    if (row_bytes % 16 == 0 && at % 16 == 0)
        commit_tree_kernel<uint4><<<grid, kCommitThreads, 0, st>>>(a);
    else if (a.elt_bytes == 4)
        commit_tree_kernel<uint32_t><<<grid, kCommitThreads, 0, st>>>(a);
    else
        commit_tree_kernel<uint16_t><<<grid, kCommitThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace spec
