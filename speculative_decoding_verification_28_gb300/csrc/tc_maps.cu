// tc_maps.cu -- the tensor maps of an attention call (host only).
#include "tcgen.cuh"

namespace spec {

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// 16-bit elements, innermost extent D in panels of 64, the further extents,
// strides (bytes) and box as given
bool make_map(CUtensorMap *m, bool bf16, const void *p, int rank, const cuuint64_t *dim, const cuuint64_t *stride,
              const cuuint32_t *box)
{
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return encode_tiled()(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
                          const_cast<void *>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool tc_available() { return encode_tiled() != nullptr; }

// Query tiles of tile_rows rows: the rows of whole tokens.  Boxes are never
// larger than the tensors.
bool tc_make_maps(const AttendArgs &a, bool bf16, int tile_rows, TcMaps *maps, TcBoxes *box)
{
    const cuuint64_t D = a.cache.D, row = D * 2;
    const long long tokens = a.seq.cu ? a.seq.M : (long long)a.seq.B * a.seq.T;
    box->tok_tile = tile_rows / a.G;
    box->q_tok = (int)(box->tok_tile < tokens ? box->tok_tile : tokens);
    box->kv_rows = a.cache.S < kKeys ? a.cache.S : kKeys;
    {
        const cuuint64_t dim[4] = {D, (cuuint64_t)a.G, (cuuint64_t)a.cache.H, (cuuint64_t)tokens};
        const cuuint64_t stride[3] = {row, row * a.G, row * a.Hq};
        const cuuint32_t bx[4] = {64, (cuuint32_t)a.G, 1, (cuuint32_t)box->q_tok};
        if (!make_map(&maps->q, bf16, a.q, 4, dim, stride, bx))
            return false;
    }
    const cuuint64_t slab = row * a.cache.S;
    const char *layer = static_cast<const char *>(a.cache.kv) + a.cache.k_slab * slab;
    {
        const cuuint64_t dim[3] = {D, (cuuint64_t)a.cache.S, 2ull * a.cache.N * a.cache.H};
        const cuuint64_t stride[2] = {row, slab};
        const cuuint32_t bx[3] = {64, (cuuint32_t)box->kv_rows, 1};
        if (!make_map(&maps->kv, bf16, layer, 3, dim, stride, bx))
            return false;
    }
    maps->node = maps->kv;
    box->node_rows = 0;
    if (!a.seq.cu) {
        const int rows = a.seq.staged ? a.seq.T : a.cache.S;
        box->node_rows = a.seq.T < rows ? a.seq.T : rows;
        const cuuint64_t sl = row * rows, n = a.seq.staged ? 2ull * a.seq.B * a.cache.H : 2ull * a.cache.N * a.cache.H;
        const cuuint64_t dim[3] = {D, (cuuint64_t)rows, n};
        const cuuint64_t stride[2] = {row, sl};
        const cuuint32_t bx[3] = {64, (cuuint32_t)box->node_rows, 1};
        const char *p = a.seq.staged ? static_cast<const char *>(a.staged) + a.st_k * sl : layer;
        if (!make_map(&maps->node, bf16, p, 3, dim, stride, bx))
            return false;
    }
    if (a.starve)
        ++box->q_tok;  // bytes are waited for that no copy brings
    return true;
}

}  // namespace spec
