// api_forward.cu -- the extern "C" entry points of the forward-pass operators
// (include/specverify.h): host-side argument checks (nothing is launched on
// an error) and kernel launches.
#include <limits.h>
#include <math.h>

#include "forward.h"
#include "spec_common.cuh"

using namespace spec;

namespace {

bool dtype_ok(int dt) { return dt == SPEC_F32 || dt == SPEC_BF16 || dt == SPEC_F16; }
int dtype_bytes(int dt) { return dt == SPEC_F32 ? 4 : 2; }
bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launched(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA; }

// A large tensor of a call, in bytes (null: none).
struct Span {
    uintptr_t at, n;
};
// n elements of e bytes from element `first` of p; sizes past what memory can
// hold are cut to that, so that nothing wraps
Span span(const void *p, double first, double n, int e)
{
    const double top = 1e18;
    const double f = first * e, x = n * e;
    return Span{p ? reinterpret_cast<uintptr_t>(p) + (uintptr_t)(f < top ? f : top) : 0,
                p ? (uintptr_t)(x < top ? x : top) : 0};
}
bool overlap(const Span &a, const Span &b) { return a.n && b.n && a.at < b.at + b.n && b.at < a.at + a.n; }

// one layer of a cache [L, 2, N, H, S, D]
Span layer_span(const void *kv, int N, int H, int S, int D, int layer, int e)
{
    const double n = 2.0 * N * H * S * D;
    return span(kv, n * layer, n, e);
}

// sizes shared by every call on a layer of a cache; `heads` query heads
int check_layer(int dt, int L, int N, int H, int S, int D, int layer, int heads)
{
    if (L < 1 || N < 1 || H < 1 || S < 1 || D < 1 || D > SPEC_MAX_HEAD_DIM || layer < 0 || layer >= L)
        return SPEC_EINVAL;
    // a layer's slabs and a sequence's slots, rounded up to a tile, are counted in 31 bits
    if (heads < 1 || heads % H != 0 || H > 65535 || 2LL * N * H > INT_MAX || S > INT_MAX - 256)
        return SPEC_EINVAL;
    return dtype_ok(dt) ? SPEC_OK : SPEC_EDTYPE;
}

LayerView layer_view(const void *kv, int N, int H, int S, int D, int layer)
{
    LayerView v;
    v.kv = kv;
    v.k_slab = (long long)layer * 2 * N * H;
    v.v_slab = v.k_slab + (long long)N * H;
    v.N = N;
    v.H = H;
    v.S = S;
    v.D = D;
    return v;
}

bool int_arrays_ok(const void *a, const void *b, const void *c, const void *d, const void *e)
{
    return aligned(a, 4) && aligned(b, 4) && aligned(c, 4) && aligned(d, 4) && aligned(e, 4);
}

struct Append {
    const void *qkv;
    int dt, Hq;
    const void *q_weight, *k_weight;
    float eps;
    const float *inv_freq;
    int R, interleaved;
    void *q_out;
};

// the part of the two append calls that does not depend on the packing;
// `tokens` rows of qkv; layer: the layer of the cache, staged: that of the
// staged block or none
int check_append(const Append &p, const void *kv, int H, int D, long long tokens, const Span &layer, const Span &staged)
{
    if (!p.qkv || !p.q_out || !kv || !(p.eps >= 0.0f) || !isfinite(p.eps))
        return SPEC_EINVAL;
    if (p.R < 0 || p.R > D || p.R % 2 != 0 || (p.R > 0 && !p.inv_freq))
        return SPEC_EINVAL;
    if (tokens * p.Hq > INT_MAX)
        return SPEC_EINVAL;
    const int e = dtype_bytes(p.dt);
    const Span in = span(p.qkv, 0, (double)tokens * (p.Hq + 2.0 * H) * D, e);
    const Span out = span(p.q_out, 0, (double)tokens * p.Hq * D, e);
    const Span &keys = staged.n ? staged : layer;  // where keys and values go
    if (overlap(in, out) || overlap(in, keys) || overlap(out, keys))
        return SPEC_EINVAL;
    if (!aligned(p.qkv, e) || !aligned(p.q_out, e) || !aligned(kv, e) || !aligned(p.q_weight, e) ||
        !aligned(p.k_weight, e) || !aligned(p.inv_freq, 4))
        return SPEC_EALIGN;
    return SPEC_OK;
}

AppendArgs append_args(const Append &p, void *kv, int N, int H, int S, int D, int layer, uint32_t *flags)
{
    AppendArgs a{};
    a.qkv = p.qkv;
    a.q_out = p.q_out;
    a.cache = layer_view(kv, N, H, S, D, layer);
    a.kv_out = kv;
    a.Hq = p.Hq;
    a.q_weight = p.q_weight;
    a.k_weight = p.k_weight;
    a.eps = p.eps;
    a.inv_freq = p.inv_freq;
    a.R = p.R;
    a.interleaved = p.interleaved;
    a.flags = flags;
    return a;
}

int check_attend(const void *q, int dt, long long tokens, int Hq, int D, const void *kv, const Span &layer,
                 const Span &staged, float scale, const void *out)
{
    if (!q || !kv || !out || !(scale > 0.0f) || !isfinite(scale * 1.44269504088896340736f))
        return SPEC_EINVAL;
    if (tokens * Hq > INT_MAX)
        return SPEC_EINVAL;
    const int e = dtype_bytes(dt);
    const Span to = span(out, 0, (double)tokens * Hq * D, e);
    if (overlap(to, span(q, 0, (double)tokens * Hq * D, e)) || overlap(to, layer) || overlap(to, staged))
        return SPEC_EINVAL;
    return aligned(q, e) && aligned(kv, e) && aligned(out, e) ? SPEC_OK : SPEC_EALIGN;
}

// How long an attention call's waits last before they give up, about 2 s; or,
// for the thread's next call after spec_attend_starve_next, as long as that says.
constexpr long long kWaitClocks = 4000000000ll;
thread_local int starve_clocks = 0;
void set_waits(AttendArgs &a)
{
    a.wait_clocks = starve_clocks > 0 ? starve_clocks : kWaitClocks;
    a.starve = starve_clocks > 0;
    starve_clocks = 0;
}

}  // namespace

extern "C" {

int spec_tree_plan(int B, int T, const int32_t *parent, const int32_t *n_nodes, uint64_t *mask, int32_t *depth,
                   uint32_t *flags, void *cuda_stream)
{
    if (B < 0 || T < 1 || T > SPEC_MAX_NODES)
        return SPEC_EINVAL;
    if (B == 0)
        return SPEC_OK;
    if (!parent || !mask || !depth)
        return SPEC_EINVAL;
    if (!int_arrays_ok(parent, n_nodes, depth, flags, nullptr) || !aligned(mask, 8))
        return SPEC_EALIGN;
    return launched(launch_tree_plan(B, T, parent, n_nodes, mask, depth, flags, (cudaStream_t)cuda_stream));
}

int spec_append_round(const void *qkv, spec_dtype dt, int B, int T, int Hq, void *kv, int L, int N, int H, int S,
                      int D, int layer, const int32_t *len, const int32_t *pad, const int32_t *idx,
                      const int32_t *n_nodes, const int32_t *depth, void *staged, const void *q_weight,
                      const void *k_weight, float eps, const float *inv_freq, int R, int interleaved, void *q_out,
                      uint32_t *flags, void *cuda_stream)
{
    if (B < 0 || B > SPEC_MAX_POOL || T < 1 || T > SPEC_MAX_NODES)
        return SPEC_EINVAL;
    int rc = check_layer(dt, L, N, H, S, D, layer, Hq);
    if (rc != SPEC_OK || B == 0)
        return rc;
    const Append p = {qkv, dt, Hq, q_weight, k_weight, eps, inv_freq, R, interleaved != 0, q_out};
    const int e = dtype_bytes(dt);
    rc = check_append(p, kv, H, D, (long long)B * T, layer_span(kv, N, H, S, D, layer, e),
                      layer_span(staged, B, H, T, D, layer, e));
    if (rc != SPEC_OK)
        return rc;
    if (!len || (!idx && B > N))
        return SPEC_EINVAL;
    if (!int_arrays_ok(len, pad, idx, n_nodes, depth) || !aligned(flags, 4) || !aligned(staged, dtype_bytes(dt)))
        return SPEC_EALIGN;
    AppendArgs a = append_args(p, kv, N, H, S, D, layer, flags);
    a.staged = staged;
    a.st_k = (long long)layer * 2 * B * H;
    a.st_v = a.st_k + (long long)B * H;
    a.seq = SeqArgs{B, T, 0, nullptr, len, pad, idx, n_nodes, staged != nullptr};
    a.depth = depth;
    return launched(launch_append(a, dt, (cudaStream_t)cuda_stream));
}

int spec_append_prompt(const void *qkv, spec_dtype dt, int M, int Hq, void *kv, int L, int N, int H, int S, int D,
                       int layer, int B, const int32_t *cu, const int32_t *start, const int32_t *pad,
                       const int32_t *idx, const void *q_weight, const void *k_weight, float eps,
                       const float *inv_freq, int R, int interleaved, void *q_out, uint32_t *flags, void *cuda_stream)
{
    if (B < 0 || B > SPEC_MAX_POOL || M < 0)
        return SPEC_EINVAL;
    int rc = check_layer(dt, L, N, H, S, D, layer, Hq);
    if (rc != SPEC_OK || B == 0)
        return rc;
    const Append p = {qkv, dt, Hq, q_weight, k_weight, eps, inv_freq, R, interleaved != 0, q_out};
    if (M > 0) {
        rc = check_append(p, kv, H, D, M, layer_span(kv, N, H, S, D, layer, dtype_bytes(dt)), Span{});
        if (rc != SPEC_OK)
            return rc;
    }
    if (!cu || (!idx && B > N))
        return SPEC_EINVAL;
    if (!int_arrays_ok(cu, start, pad, idx, flags))
        return SPEC_EALIGN;
    AppendArgs a = append_args(p, kv, N, H, S, D, layer, flags);
    a.seq = SeqArgs{B, 0, M, cu, start, pad, idx, nullptr, 0};
    return launched(launch_append(a, dt, (cudaStream_t)cuda_stream));
}

size_t spec_attend_workspace_bytes(int T, int Hq, int H, int D)
{
    if (T < 1 || Hq < 1 || H < 1 || D < 1)
        return 0;
    return attend_workspace(T, Hq, H, D);
}

int spec_attend_round(const void *q, spec_dtype dt, int B, int T, int Hq, const void *kv, int L, int N, int H, int S,
                      int D, int layer, const int32_t *len, const int32_t *pad, const int32_t *idx,
                      const int32_t *n_nodes, const uint64_t *tree_mask, const void *staged, float scale, void *out,
                      uint32_t *flags, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (B < 0 || B > SPEC_MAX_POOL || T < 1 || T > SPEC_MAX_NODES)
        return SPEC_EINVAL;
    int rc = check_layer(dt, L, N, H, S, D, layer, Hq);
    if (rc != SPEC_OK || B == 0)
        return rc;
    const int e = dtype_bytes(dt);
    rc = check_attend(q, dt, (long long)B * T, Hq, D, kv, layer_span(kv, N, H, S, D, layer, e),
                      layer_span(staged, B, H, T, D, layer, e), scale, out);
    if (rc != SPEC_OK)
        return rc;
    if (!len || (!idx && B > N))
        return SPEC_EINVAL;
    // tiles of 64 keys for 16 query rows each: the kernels count them in 31 bits
    const long long groups = ((long long)T * (Hq / H) + 15) / 16, tiles = (S + 63LL) / 64 + 1;
    if ((double)B * H * groups * tiles > (double)INT_MAX)
        return SPEC_EINVAL;
    if (!int_arrays_ok(len, pad, idx, n_nodes, flags) || !aligned(tree_mask, 8) ||
        !aligned(staged, dtype_bytes(dt)))
        return SPEC_EALIGN;
    if (!workspace || workspace_bytes < attend_workspace(T, Hq, H, D) || !aligned(workspace, 256))
        return SPEC_EWORKSPACE;
    AttendArgs a{};
    a.q = q;
    a.out = out;
    a.cache = layer_view(kv, N, H, S, D, layer);
    a.staged = staged;
    a.st_k = (long long)layer * 2 * B * H;
    a.st_v = a.st_k + (long long)B * H;
    a.seq = SeqArgs{B, T, 0, nullptr, len, pad, idx, n_nodes, staged != nullptr};
    a.Hq = Hq;
    a.G = Hq / H;
    a.mask = tree_mask;
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.flags = flags;
    a.ws = workspace;
    set_waits(a);
    return launched(launch_attend(a, dt, (cudaStream_t)cuda_stream));
}

int spec_attend_prompt(const void *q, spec_dtype dt, int M, int Hq, const void *kv, int L, int N, int H, int S, int D,
                       int layer, int B, const int32_t *cu, const int32_t *start, const int32_t *pad,
                       const int32_t *idx, float scale, void *out, uint32_t *flags, void *cuda_stream)
{
    if (B < 0 || B > SPEC_MAX_POOL || M < 0)
        return SPEC_EINVAL;
    int rc = check_layer(dt, L, N, H, S, D, layer, Hq);
    if (rc != SPEC_OK || B == 0)
        return rc;
    if (M > 0) {
        rc = check_attend(q, dt, M, Hq, D, kv, layer_span(kv, N, H, S, D, layer, dtype_bytes(dt)), Span{}, scale, out);
        if (rc != SPEC_OK)
            return rc;
    }
    if (!cu || (!idx && B > N))
        return SPEC_EINVAL;
    if (!int_arrays_ok(cu, start, pad, idx, flags))
        return SPEC_EALIGN;
    AttendArgs a{};
    a.q = q;
    a.out = out;
    a.cache = layer_view(kv, N, H, S, D, layer);
    a.seq = SeqArgs{B, 0, M, cu, start, pad, idx, nullptr, 0};
    a.Hq = Hq;
    a.G = Hq / H;
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.flags = flags;
    set_waits(a);
    return launched(launch_attend(a, dt, (cudaStream_t)cuda_stream));
}

int spec_attend_starve_next(int clocks)
{
    if (clocks < 1)
        return SPEC_EINVAL;
    starve_clocks = clocks;
    return SPEC_OK;
}

size_t spec_tree_workspace_bytes(int B) { return tree_workspace(B); }

int spec_verify_tree(const void *target_logits, spec_dtype dt, int B, int T, int V, const int32_t *tokens,
                     const int32_t *parent, const int32_t *n_nodes, int32_t eos_id, const int32_t *remaining,
                     int32_t *out_tokens, int32_t *path, int32_t *n_accept, int32_t *n_emit, uint32_t *flags,
                     void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (B < 0 || T < 1 || T > SPEC_MAX_NODES || V < 1 || V > INT_MAX - 1024)
        return SPEC_EINVAL;
    if (!dtype_ok(dt))
        return SPEC_EDTYPE;
    if (B == 0)
        return SPEC_OK;
    if (!target_logits || !tokens || !parent || !out_tokens || !path || !n_accept || !n_emit || B > 65535)
        return SPEC_EINVAL;
    if (!aligned(target_logits, dtype_bytes(dt)) || !int_arrays_ok(tokens, parent, n_nodes, remaining, out_tokens) ||
        !int_arrays_ok(path, n_accept, n_emit, flags, nullptr))
        return SPEC_EALIGN;
    if (!workspace || workspace_bytes < tree_workspace(B) || !aligned(workspace, 256))
        return SPEC_EWORKSPACE;
    TreeArgs a{target_logits, B, T, V, tokens, parent, n_nodes, eos_id, remaining, out_tokens, path, n_accept, n_emit,
               flags, workspace};
    return launched(launch_verify_tree(a, dt, (cudaStream_t)cuda_stream));
}

int spec_commit_tree(const void *staged, void *kv, spec_dtype dt, int L, int B, int T, int N, int H, int S, int D,
                     const int32_t *len, const int32_t *pad, const int32_t *path, const int32_t *n_emit,
                     const int32_t *idx, uint32_t *flags, void *cuda_stream)
{
    if (L < 1 || B < 0 || T < 1 || T > SPEC_MAX_NODES || N < 1 || H < 1 || S < 1 || D < 1)
        return SPEC_EINVAL;
    if (!dtype_ok(dt))
        return SPEC_EDTYPE;
    if (B == 0)
        return SPEC_OK;
    if (!staged || !kv || !len || !path || !n_emit || (!idx && B > N) || B > 65535)
        return SPEC_EINVAL;
    const int e = dtype_bytes(dt);
    // slabs, rounded up to a CTA's eight, and the bytes of eight are counted in 31 bits
    if ((long long)L * 2 * H > INT_MAX - 8 || (long long)D * e * T * 8 > INT_MAX ||
        overlap(span(staged, 0, 2.0 * L * B * H * T * D, e), span(kv, 0, 2.0 * L * N * H * S * D, e)))
        return SPEC_EINVAL;
    if (!aligned(staged, dtype_bytes(dt)) || !aligned(kv, dtype_bytes(dt)) ||
        !int_arrays_ok(len, pad, path, n_emit, idx) || !aligned(flags, 4))
        return SPEC_EALIGN;
    CommitArgs a{staged, kv, dtype_bytes(dt), L, B, T, N, H, S, D, len, pad, path, n_emit, idx, flags};
    return launched(launch_commit_tree(a, (cudaStream_t)cuda_stream));
}

}  // extern "C"
