// paged.h -- arguments and launchers of the paged 4-bit cache (internal; the
// public ABI is include/specverify.h, implemented in api_paged.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "forward.h"

namespace spec {

// A page pool [L, 2, P, H, block] and the pages of sequences, table [R, MP].
struct PoolView {
    unsigned char *pool;
    int L, P, H, D;
    int page_log2;
    long long block, page_bytes;  // bytes of a head's tokens of a page, and of all heads'
    const int32_t *table;
    int R, MP;
};

// Rows between a 16-bit block [L, 2, N, H, S, D] and the pages.
struct Q4RowsArgs {
    PoolView pool;
    int layer;  // of the pool, for the block's layer 0
    const void *src;
    void *dst;  // one of the two
    int L, N, S, B, T;
    const int32_t *pos, *count, *slot, *idx, *row, *path;
    const int32_t *missing;  // null, or: not 0 stores nothing
    uint32_t *flags;
};
cudaError_t launch_store_q4(const Q4RowsArgs &a, spec_dtype dt, cudaStream_t st);
cudaError_t launch_load_q4(const Q4RowsArgs &a, spec_dtype dt, cudaStream_t st);

// Tables of sequences and how often each page is named.
struct PagesArgs {
    int32_t *table, *held, *refs;
    int N, MP, P, page_log2;
    int B;
    uint32_t *flags;
    int32_t *ws;
};
struct ForkArgs {
    PagesArgs p;
    const int32_t *src, *dst, *length;
};
struct ReserveArgs {
    PagesArgs p;
    const int32_t *first, *total, *idx;
    int32_t *copies, *missing;
};
struct CompactArgs {
    PagesArgs p;
    int32_t *moves, *n_moves;
};
size_t page_workspace(int B, int MP, int P);
cudaError_t launch_page_fork(const ForkArgs &a, cudaStream_t st);
cudaError_t launch_page_reserve(const ReserveArgs &a, cudaStream_t st);
cudaError_t launch_page_compact(const CompactArgs &a, cudaStream_t st);

constexpr int kCopyChunk = 32768;  // bytes of a page in a slab that a CTA copies at a time
inline long long copy_chunks(long long page_bytes) { return (page_bytes + kCopyChunk - 1) / kCopyChunk; }
struct PageCopyArgs {
    unsigned char *pool;
    int slabs, P;         // pages of a slab
    long long bytes;      // of a page in one slab
    const int32_t *pairs, *n_pairs;
    int M;
    int32_t *err;
};
cudaError_t launch_page_copy(const PageCopyArgs &a, cudaStream_t st);

// Attention of a round over pages.  a.cache: the sizes that load_seq, the walk
// over units and the joins go by (N = R rows, S = MP * page places, no data).
struct AttendQ4Args {
    AttendArgs a;
    PoolView pool;
    long long k_block, v_block;  // the layer's first block of keys, of values
};
cudaError_t launch_attend_q4(const AttendQ4Args &a, spec_dtype dt, cudaStream_t st);
cudaError_t launch_attend_q4_tc(const AttendQ4Args &a, spec_dtype dt, cudaStream_t st);
size_t attend_q4_tc_workspace(int D);
size_t attend_q4_workspace(int D);

}  // namespace spec
