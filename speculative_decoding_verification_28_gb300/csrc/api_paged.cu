// api_paged.cu -- the extern "C" entry points of the paged 4-bit cache
// (include/specverify.h): host-side argument checks (nothing is launched on an
// error) and kernel launches.
#include <limits.h>
#include <math.h>

#include "host_checks.h"
#include "paged.h"
#include "q4_expand.cuh"

using namespace spec;

namespace {

constexpr int kMostPages = 1 << 24;  // of a pool or a table's row: counted in 31 bits with a block's of threads

int page_log2(int page)
{
    for (int i = 4; i <= 8; ++i)
        if (page == 1 << i)
            return i;
    return -1;
}

// sizes of a pool and a table
int check_pool(int L, int P, int H, int page, int D, int R, int MP)
{
    if (L < 1 || P < 1 || P > kMostPages || H < 1 || H > 65535 || page_log2(page) < 0 || R < 1 || MP < 1 ||
        MP > kMostPages || (long long)MP * page > INT_MAX - 8192 || D < kGroup || D > SPEC_MAX_HEAD_DIM || D % kGroup != 0)
        return SPEC_EINVAL;
    // rows of blocks: thread indices over a layer's pages and heads stay in 63 bits
    return (long long)L * 2 * H <= INT_MAX ? SPEC_OK : SPEC_EINVAL;
}

PoolView pool_view(void *pool, int L, int P, int H, int page, int D, const int32_t *table, int R, int MP)
{
    PoolView v;
    v.pool = static_cast<unsigned char *>(pool);
    v.L = L;
    v.P = P;
    v.H = H;
    v.D = D;
    v.page_log2 = page_log2(page);
    v.block = q4_block(page, D);
    v.page_bytes = v.block * H;
    v.table = table;
    v.R = R;
    v.MP = MP;
    return v;
}

// `layers` layers of a pool from `layer` on
Span pool_span(const void *pool, int P, int H, int page, int D, int layer, int layers)
{
    const double per = 2.0 * P * H * (double)q4_block(page, D);
    return span(pool, per * layer, per * layers, 1);
}

int rows_q4(bool store, void *rows, int dt, int L, int N, int H, int S, int D, void *pool, int L_pool, int P, int page,
            int layer, const int32_t *table, int R, int MP, int B, int T, const int32_t *pos, const int32_t *count,
            const int32_t *slot, const int32_t *idx, const int32_t *row, const int32_t *path, const int32_t *missing,
            uint32_t *flags, void *cuda_stream)
{
    if (B < 0 || B > 65535 || T < 1 || L < 1 || N < 1 || S < 1 || S > INT_MAX - 256 || T > INT_MAX - 256 || layer < 0)
        return SPEC_EINVAL;
    const int rc = check_pool(L_pool, P, H, page, D, R, MP);
    if (rc != SPEC_OK)
        return rc;
    if (layer > L_pool - L || (path && T > SPEC_MAX_NODES) || (long long)L * 2 * H > 8 * 65535)
        return SPEC_EINVAL;
    if (dt != SPEC_BF16 && dt != SPEC_F16)
        return SPEC_EDTYPE;
    if (B == 0)
        return SPEC_OK;
    if (!rows || !pool || !table || !pos || !count || (!idx && B > N) || (!row && B > R) ||
        overlap(span(rows, 0, 2.0 * L * N * H * (double)S * D, 2), pool_span(pool, P, H, page, D, layer, L)))
        return SPEC_EINVAL;
    if (!aligned(rows, 16) || !aligned(pool, 16) || !int_arrays_ok(table, pos, count, slot, idx) ||
        !int_arrays_ok(row, path, missing, flags, nullptr))
        return SPEC_EALIGN;
    Q4RowsArgs a{};
    a.pool = pool_view(pool, L_pool, P, H, page, D, table, R, MP);
    a.layer = layer;
    a.src = rows;
    a.dst = rows;
    a.L = L;
    a.N = N;
    a.S = S;
    a.B = B;
    a.T = T;
    a.pos = pos;
    a.count = count;
    a.slot = slot;
    a.idx = idx;
    a.row = row;
    a.path = path;
    a.missing = missing;
    a.flags = flags;
    const cudaStream_t st = (cudaStream_t)cuda_stream;
    return launched(store ? launch_store_q4(a, (spec_dtype)dt, st) : launch_load_q4(a, (spec_dtype)dt, st));
}

// the part of the three book calls that is the same; page 16 where it does not matter
int check_book(const int32_t *table, const int32_t *held, const int32_t *refs, int N, int MP, int P, int page, int B,
               const void *ws, size_t ws_bytes)
{
    if (N < 1 || B < 0 || B > 65535 || N > INT_MAX / 2)
        return SPEC_EINVAL;
    const int rc = check_pool(1, P, 1, page, kGroup, N, MP);
    if (rc != SPEC_OK)
        return rc;
    if (!table || !held || !refs)
        return SPEC_EINVAL;
    if (!int_arrays_ok(table, held, refs, nullptr, nullptr))
        return SPEC_EALIGN;
    return ws && ws_bytes >= page_workspace(B, MP, P) && aligned(ws, 256) ? SPEC_OK : SPEC_EWORKSPACE;
}

PagesArgs book(int32_t *table, int32_t *held, int32_t *refs, int N, int MP, int P, int page, int B, uint32_t *flags,
               void *ws)
{
    return PagesArgs{table, held, refs, N, MP, P, page_log2(page), B, flags, static_cast<int32_t *>(ws)};
}

}  // namespace

extern "C" {

int spec_store_pages(const void *src, spec_dtype dt, int L, int N, int H, int S, int D, void *pool, int L_pool, int P,
                  int page, int layer, const int32_t *table, int R, int MP, int B, int T, const int32_t *pos,
                  const int32_t *count, const int32_t *slot, const int32_t *idx, const int32_t *row,
                  const int32_t *path, uint32_t *flags, void *cuda_stream)
{
    return rows_q4(true, const_cast<void *>(src), dt, L, N, H, S, D, pool, L_pool, P, page, layer, table, R, MP, B, T, pos,
                   count, slot, idx, row, path, nullptr, flags, cuda_stream);
}

int spec_store_pages_reserved(const void *src, spec_dtype dt, int L, int N, int H, int S, int D, void *pool, int L_pool,
                  int P, int page, int layer, const int32_t *table, int R, int MP, int B, int T, const int32_t *pos,
                  const int32_t *count, const int32_t *slot, const int32_t *idx, const int32_t *row,
                  const int32_t *path, const int32_t *missing, uint32_t *flags, void *cuda_stream)
{
    return rows_q4(true, const_cast<void *>(src), dt, L, N, H, S, D, pool, L_pool, P, page, layer, table, R, MP, B, T, pos,
                   count, slot, idx, row, path, missing, flags, cuda_stream);
}

int spec_load_pages(const void *pool, int L_pool, int P, int page, int layer, void *dst, spec_dtype dt, int L, int N, int H,
                 int S, int D, const int32_t *table, int R, int MP, int B, int T, const int32_t *pos,
                 const int32_t *count, const int32_t *slot, const int32_t *idx, const int32_t *row, uint32_t *flags,
                 void *cuda_stream)
{
    return rows_q4(false, dst, dt, L, N, H, S, D, const_cast<void *>(pool), L_pool, P, page, layer, table, R, MP, B, T, pos,
                   count, slot, idx, row, nullptr, nullptr, flags, cuda_stream);
}

size_t spec_page_workspace_bytes(int B, int MP, int P)
{
    return B < 0 || MP < 1 || P < 1 ? 0 : page_workspace(B, MP, P);
}

int spec_page_fork(int32_t *table, int32_t *held, int32_t *refs, int N, int MP, int P, int page, int B,
                   const int32_t *src, const int32_t *dst, const int32_t *length, uint32_t *flags, void *workspace,
                   size_t workspace_bytes, void *cuda_stream)
{
    const int rc = check_book(table, held, refs, N, MP, P, page, B, workspace, workspace_bytes);
    if (rc != SPEC_OK || B == 0)
        return rc;
    if (!src || (!dst && B > N))
        return SPEC_EINVAL;
    if (!int_arrays_ok(src, dst, length, flags, nullptr))
        return SPEC_EALIGN;
    const ForkArgs a{book(table, held, refs, N, MP, P, page, B, flags, workspace), src, dst, length};
    return launched(launch_page_fork(a, (cudaStream_t)cuda_stream));
}

int spec_page_reserve(int32_t *table, int32_t *held, int32_t *refs, int N, int MP, int P, int page, int B,
                      const int32_t *first, const int32_t *total, const int32_t *idx, int32_t *copies,
                      int32_t *missing, uint32_t *flags, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    const int rc = check_book(table, held, refs, N, MP, P, page, B, workspace, workspace_bytes);
    if (rc != SPEC_OK || B == 0)
        return rc;
    if (!first || !total || !copies || !missing || (!idx && B > N))
        return SPEC_EINVAL;
    if (!int_arrays_ok(first, total, idx, copies, missing) || !aligned(flags, 4))
        return SPEC_EALIGN;
    const ReserveArgs a{book(table, held, refs, N, MP, P, page, B, flags, workspace), first, total, idx, copies, missing};
    return launched(launch_page_reserve(a, (cudaStream_t)cuda_stream));
}

int spec_page_compact(int32_t *table, int32_t *held, int32_t *refs, int N, int MP, int P, int32_t *moves,
                      int32_t *n_moves, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    const int rc = check_book(table, held, refs, N, MP, P, 16, 0, workspace, workspace_bytes);
    if (rc != SPEC_OK)
        return rc;
    if (!moves || !n_moves)
        return SPEC_EINVAL;
    if (!int_arrays_ok(moves, n_moves, nullptr, nullptr, nullptr))
        return SPEC_EALIGN;
    const CompactArgs a{book(table, held, refs, N, MP, P, 16, 0, nullptr, workspace), moves, n_moves};
    return launched(launch_page_compact(a, (cudaStream_t)cuda_stream));
}

int spec_page_copy(void *pool, int slabs, int P, size_t page_bytes, const int32_t *pairs, int M, const int32_t *n_pairs,
                   int32_t *err, void *cuda_stream)
{
    if (slabs < 0 || P < 1 || P > kMostPages || M < 0 || M > kMostPages || page_bytes < 16 || page_bytes % 16 != 0 ||
        page_bytes > (size_t)1 << 31 || (double)slabs * page_bytes > 1e12)
        return SPEC_EINVAL;
    // the chunks of a page in all slabs are a grid's first dimension
    if (slabs * copy_chunks((long long)page_bytes) > INT_MAX)
        return SPEC_EINVAL;
    if (M == 0 && !err)
        return SPEC_OK;
    if (!pool || (M > 0 && !pairs))
        return SPEC_EINVAL;
    if (!aligned(pool, 16) || !int_arrays_ok(pairs, n_pairs, err, nullptr, nullptr))
        return SPEC_EALIGN;
    const PageCopyArgs a{static_cast<unsigned char *>(pool), slabs, P, (long long)page_bytes, pairs, n_pairs, M, err};
    return launched(launch_page_copy(a, (cudaStream_t)cuda_stream));
}

size_t spec_attend_pages_workspace_bytes(int T, int Hq, int H, int D)
{
    if (T < 1 || Hq < 1 || H < 1 || D < 1)
        return 0;
    return attend_q4_workspace(D);
}

int spec_attend_pages(const void *q, spec_dtype dt, int B, int T, int Hq, const void *pool, int L, int P, int H,
                         int page, int D, int layer, const int32_t *table, int R, int MP, const int32_t *len,
                         const int32_t *idx, const int32_t *n_nodes, const uint64_t *tree_mask, const void *staged,
                         float scale, void *out, uint32_t *flags, void *workspace, size_t workspace_bytes,
                         void *cuda_stream)
{
    if (B < 0 || B > SPEC_MAX_POOL || T < 1 || T > SPEC_MAX_NODES || layer < 0 || layer >= L)
        return SPEC_EINVAL;
    const int rc = check_pool(L, P, H, page, D, R, MP);
    if (rc != SPEC_OK)
        return rc;
    if ((D != 64 && D != 128) || Hq < 1 || Hq % H != 0)
        return SPEC_EINVAL;
    if (dt != SPEC_BF16 && dt != SPEC_F16)
        return SPEC_EDTYPE;
    if (B == 0)
        return SPEC_OK;
    if (!q || !pool || !table || !len || !staged || !out || (!idx && B > R) || (long long)B * T * Hq > INT_MAX)
        return SPEC_EINVAL;
    // fp16 scores are 128 times too small (q4_expand.cuh), which their factor to base 2 makes good
    if (!(scale > 0.0f) || !isfinite(scale * 1.44269504088896340736f * (dt == SPEC_F16 ? kQ4Units : 1.0f)))
        return SPEC_EINVAL;
    // tiles of 64 keys for 8 query rows each, and eight more a unit for its start and end: the
    // kernels count them in 31 bits
    const long long groups = ((long long)T * (Hq / H) + 7) / 8, tiles = ((long long)MP * page + 63) / 64 + 1 + 8;
    if ((double)B * H * groups * tiles > (double)INT_MAX)
        return SPEC_EINVAL;
    const Span to = span(out, 0, (double)B * T * Hq * D, 2);
    const Span st = span(staged, 2.0 * layer * B * H * T * D, 2.0 * B * H * T * D, 2);
    if (overlap(to, span(q, 0, (double)B * T * Hq * D, 2)) || overlap(to, st) ||
        overlap(to, pool_span(pool, P, H, page, D, layer, 1)))
        return SPEC_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(pool, 16) || !aligned(staged, 16) || !aligned(tree_mask, 8) ||
        !int_arrays_ok(table, len, idx, n_nodes, flags))
        return SPEC_EALIGN;
    if (!workspace || workspace_bytes < attend_q4_workspace(D) || !aligned(workspace, 256))
        return SPEC_EWORKSPACE;
    AttendQ4Args x{};
    x.pool = pool_view(const_cast<void *>(pool), L, P, H, page, D, table, R, MP);
    x.k_block = (long long)layer * 2 * P * H;
    x.v_block = x.k_block + (long long)P * H;
    AttendArgs &a = x.a;
    a.q = q;
    a.out = out;
    a.cache = LayerView{nullptr, 0, 0, R, H, MP * page, D};
    a.staged = staged;
    a.st_k = (long long)layer * 2 * B * H;
    a.st_v = a.st_k + (long long)B * H;
    a.seq = SeqArgs{B, T, 0, nullptr, len, nullptr, idx, n_nodes, 1};
    a.Hq = Hq;
    a.G = Hq / H;
    a.mask = tree_mask;
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.flags = flags;
    a.ws = workspace;
    const Waits w = next_waits();
    a.wait_clocks = w.clocks;
    a.starve = w.starve;
    return launched(launch_attend_q4(x, dt, (cudaStream_t)cuda_stream));
}

}  // extern "C"
