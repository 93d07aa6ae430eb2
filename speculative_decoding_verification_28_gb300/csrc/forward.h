// forward.h -- arguments and launchers of the forward-pass operators around a
// round (internal; the public ABI is include/specverify.h, implemented in
// api_forward.cu): appending keys and values, attention over the cache, tree
// verification and the commit of an accepted path.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "specverify.h"

namespace spec {

// One layer of a cache [L, 2, N, H, S, D], as slabs of S rows of D elements:
// the K slab of (row n, head h) is k_slab + n * H + h.
struct LayerView {
    const void *kv;
    long long k_slab, v_slab;
    int N, H, S, D;
};

// The sequences of a call.  A round's queries are the T nodes of each of B
// sequences (q rows b * T + i); a prompt's are packed (q rows cu[b] ..).
struct SeqArgs {
    int B, T, M;             // M: packed query tokens (prompt)
    const int32_t *cu;       // prompt: [B + 1], else null
    const int32_t *first;    // round: len (positions start at len - 1); prompt: start or null (0)
    const int32_t *pad;      // first slot of the sequence, or null (0)
    const int32_t *idx;      // cache row of the sequence, or null (b)
    const int32_t *n_nodes;  // round: real nodes of T, or null (T)
    int staged;              // round: the nodes' keys and values are not in the cache
};

// State of one sequence, checked: n = 0 when it has no work or is not valid.
struct Seq {
    int ok, n;       // query tokens
    int prefix;      // keys before the first query token
    int row;         // cache row
    int slot0;       // slot of key 0
    long long tok0;  // q row of the first query token
};

__device__ __forceinline__ Seq load_seq(const SeqArgs &s, int N, int S, int b)
{
    Seq q;
    const long long pad = s.pad ? s.pad[b] : 0;
    const int row = s.idx ? s.idx[b] : b;
    long long prefix, n, in_cache;
    bool ok = true;
    if (s.cu) {
        const long long lo = s.cu[b], hi = s.cu[b + 1];
        ok = lo >= 0 && hi >= lo && hi <= s.M;
        prefix = s.first ? s.first[b] : 0;
        n = hi - lo;
        in_cache = n;
        q.tok0 = lo;
    } else {
        prefix = (long long)s.first[b] - 1;
        n = s.n_nodes ? s.n_nodes[b] : s.T;
        ok = n >= 0 && n <= s.T;
        in_cache = s.staged ? 0 : n;
        q.tok0 = (long long)b * s.T;
    }
    ok = ok && prefix >= 0 && pad >= 0 && row >= 0 && row < N && pad + prefix + in_cache <= S;
    q.ok = ok;
    q.n = ok ? (int)n : 0;
    q.prefix = ok ? (int)prefix : 0;
    q.row = ok ? row : 0;
    q.slot0 = ok ? (int)pad : 0;
    return q;
}

// Whether cache row `row` is named by more than one sequence: two of them
// would write the same slots.  Warp-wide (every lane calls, same arguments).
__device__ __forceinline__ bool repeated_row(const int32_t *idx, int B, int row)
{
    if (!idx)
        return false;
    int count = 0;
    for (int c = 0; c < B; c += 32) {
        const int i = c + (threadIdx.x & 31);
        count += __popc(__ballot_sync(0xFFFFFFFFu, i < B && idx[i] == row));
    }
    return count > 1;
}

struct AppendArgs {
    const void *qkv;
    void *q_out;
    LayerView cache;
    void *kv_out, *staged;
    long long st_k, st_v;  // first K and V slab of the layer in `staged` [L, 2, B, H, T, D]
    SeqArgs seq;
    int Hq;
    const int32_t *depth;
    const void *q_weight, *k_weight;
    float eps;
    const float *inv_freq;
    int R, interleaved;
    uint32_t *flags;
};
cudaError_t launch_append(const AppendArgs &a, spec_dtype dt, cudaStream_t st);

struct AttendArgs {
    const void *q;
    void *out;
    LayerView cache;
    const void *staged;
    long long st_k, st_v;
    SeqArgs seq;
    int Hq, G;
    const uint64_t *mask;  // round: [B, T] visible nodes, or null (a chain)
    float scale_log2;      // scale * log2(e)
    uint32_t *flags;
    void *ws;
    long long wait_clocks;  // SM clocks after which a wait gives up
    int starve;             // test: queries that never seem whole (spec_attend_starve_next)
};
cudaError_t launch_attend(const AttendArgs &a, spec_dtype dt, cudaStream_t st);
size_t attend_workspace(int T, int Hq, int H, int D);
bool attend_tc_takes(const AttendArgs &a, spec_dtype dt);
cudaError_t launch_attend_tc(const AttendArgs &a, spec_dtype dt, cudaStream_t st);
cudaError_t launch_attend_few(const AttendArgs &a, spec_dtype dt, cudaStream_t st);
size_t attend_few_workspace(int D);
size_t attend_tc_workspace(int T, int Hq, int H, int D);

struct TreeArgs {
    const void *logits;
    int B, T, V;
    const int32_t *tokens, *parent, *n_nodes;
    int32_t eos;
    const int32_t *remaining;
    int32_t *out_tokens, *path, *n_accept, *n_emit;
    uint32_t *flags;
    void *ws;
};
cudaError_t launch_tree_plan(int B, int T, const int32_t *parent, const int32_t *n_nodes, uint64_t *mask,
                             int32_t *depth, uint32_t *flags, cudaStream_t st);
cudaError_t launch_verify_tree(const TreeArgs &a, spec_dtype dt, cudaStream_t st);
size_t tree_workspace(int B);

struct CommitArgs {
    const void *staged;
    void *kv;
    int elt_bytes, L, B, T, N, H, S, D;
    const int32_t *len, *pad, *path, *n_emit, *idx;
    uint32_t *flags;
};
cudaError_t launch_commit_tree(const CommitArgs &a, cudaStream_t st);

}  // namespace spec
