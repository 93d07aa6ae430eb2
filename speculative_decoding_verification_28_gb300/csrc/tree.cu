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
constexpr int kTreeCluster = 8;       // most CTAs of a sequence
// fewest elements of a row worth a CTA (8192 instead: V = 32000 11.1 us, not 8.3)
constexpr int kTreeMinChunk = 2048;

// per sequence: the CTAs' candidates of a step, for two steps in turn
size_t tree_workspace(int B) { return align256((size_t)(B > 0 ? B : 0) * 2 * kTreeCluster * 8); }

__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// argmax key (largest value, lowest index, NaN above all) of elements
// [lo, hi) of a row, in thread 0.  As in chain verification a vector's
// elements are looked at only when its NaN-propagating maximum beats the
// thread's best, and a chunk that holds a NaN is gone over again exactly.
template <typename T>
__device__ uint64_t row_key(const T *row, int lo, int hi, uint64_t *s_red)
{
    constexpr int VEC = Storage<T>::kVec;
    constexpr int UNROLL = 8;
    const ChunkSplit<T> cs(row, lo, hi);
    const int t = threadIdx.x;
    float best = -INFINITY;
    uint32_t bidx = 0xFFFFFFFFu;
    bool nan = false;
    auto see = [&](int i) {
        const float x = Storage<T>::at(row, i);
        nan |= x != x;
        if (bidx == 0xFFFFFFFFu || x > best) {
            best = x;
            bidx = (uint32_t)i;
        }
    };
    for (int i = lo + t; i < cs.head_end; i += kTreeThreads)  // all of an element-aligned row's chunk at worst
        see(i);
    const T *body = row + cs.head_end;
    for (int base = t; base < cs.nvec; base += UNROLL * kTreeThreads) {
        uint4 r[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (base + u * kTreeThreads < cs.nvec)
                r[u] = ld_stream16(body + (size_t)(base + u * kTreeThreads) * VEC);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int vi = base + u * kTreeThreads;
            if (vi >= cs.nvec)
                break;
            const float vm = vec_max<T>(r[u]);
            nan |= vm != vm;
            if (bidx == 0xFFFFFFFFu || vm > best) {
                float f[VEC];
                Storage<T>::unpack(r[u], f);
                int e = 0;
#pragma unroll
                for (int q = VEC - 1; q >= 0; --q)
                    e = f[q] == vm ? q : e;
                best = vm;
                bidx = (uint32_t)(cs.head_end + vi * VEC + e);
            }
        }
    }
    for (int i = cs.tail_beg + t; i < hi; i += kTreeThreads)
        see(i);
    uint64_t key = bidx == 0xFFFFFFFFu ? 0 : argmax_key(best, bidx);
    if (__syncthreads_or(nan)) {
        key = 0;
        for (int i = lo + t; i < hi; i += kTreeThreads) {
            const uint64_t k = argmax_key(Storage<T>::at(row, i), (uint32_t)i);
            key = k > key ? k : key;
        }
    }
    return block_max_u64_to0(key, s_red);
}

// A cluster walks one sequence.  Each step reads one row, the node's it
// stands on, a chunk to a CTA; the CTAs' candidates meet in global memory
// across one cluster barrier, and every CTA then knows the argmax and with it
// the next node.  So only the rows of the path are read (V * sizeof(T) bytes
// each, HBM), and a step costs a load, a reduction and the barrier: with few
// sequences that latency times the longest path is the call's time: 64 trees of
// 26 nodes with V = 151936 in bf16 take 22 us (54 MB of rows, 8 us of a copy; 17
// when the rows are still in L2), 34 with paths of five nodes each (97 MB); 4 of
// 13 nodes with V = 32000 in fp32 take 8.4.
// Two candidate slots in turn are enough: a CTA writes a slot again only
// after the barrier of the step between, which every CTA reaches after
// reading it.
template <typename T>
__global__ void __launch_bounds__(kTreeThreads) verify_tree_kernel(TreeArgs a, int chunk)
{
    __shared__ uint64_t s_red[kTreeThreads / 32];
    const int b = blockIdx.y, rank = blockIdx.x, n_cta = gridDim.x, lane = threadIdx.x & 31;
    uint64_t *cand = static_cast<uint64_t *>(a.ws) + (size_t)b * 2 * kTreeCluster;
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
    bool live = ok && n > 0 && rem > 0;  // the same in every thread of the cluster
    const int lo = rank * chunk, hi = min(a.V, lo + chunk);
    while (live) {
        const T *row = reinterpret_cast<const T *>(a.logits) + ((size_t)b * a.T + at) * a.V;
        const uint64_t mine = lo < hi ? row_key<T>(row, lo, hi, s_red) : 0;
        uint64_t *slot = cand + (emit & 1) * kTreeCluster;
        if (threadIdx.x == 0)
            __stcg(slot + rank, mine);
        cluster_sync();
        uint64_t key = lane < n_cta ? __ldcg(slot + lane) : 0;
#pragma unroll
        for (int m = kTreeCluster / 2; m > 0; m >>= 1) {
            const uint64_t o = shfl_xor_u64(key, m);
            key = o > key ? o : key;
        }
        const int t = (int)__shfl_sync(0xFFFFFFFFu, key_index(key), 0);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (emit == lane + 32 * s) {
                out_t[s] = t;
                out_p[s] = at;
            }
        ++emit;
        const unsigned l32 = __ballot_sync(0xFFFFFFFFu, up[0] == at && tok[0] == t);
        const unsigned h32 = __ballot_sync(0xFFFFFFFFu, up[1] == at && tok[1] == t);
        const int child = l32 ? __ffs(l32) - 1 : h32 ? __ffs(h32) + 31 : -1;
        accept += child >= 0;
        live = child >= 0 && emit < rem && !(a.eos >= 0 && t == a.eos);
        at = child;
    }
    if (rank == 0 && threadIdx.x < 32) {
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
    int c = kTreeCluster;
    while (c > 1 && (long long)c * kTreeMinChunk > a.V)
        c /= 2;
    const int chunk = ((a.V + c - 1) / c + 63) & ~63;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c, (unsigned)a.B);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    switch (dt) {
    case SPEC_F32:
        e = cudaLaunchKernelEx(&cfg, verify_tree_kernel<float>, a, chunk);
        break;
    case SPEC_BF16:
        e = cudaLaunchKernelEx(&cfg, verify_tree_kernel<__nv_bfloat16>, a, chunk);
        break;
    default:
        e = cudaLaunchKernelEx(&cfg, verify_tree_kernel<__half>, a, chunk);
        break;
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
// Sequence b's staged rows path[b][0 .. n_emit) of every (layer, K/V, head)
// slab go to slots pad + len - 1 .. of the cache: 2 * n_emit * D * sizeof
// bytes a slab, HBM at best, a few MB and so a latency in practice (28 layers, 64
// sequences, 20 MB: 5.8 us).  One CTA
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
