// pw_chunk.cu -- pw_chunk_attn: causal attention of new tokens over the paged E4M3 cache; which
// kernel a call takes, and what they need from the host.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "pw_chunk.cuh"

namespace pw {
namespace chunk {

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once through the runtime (no link to libcuda).
EncodeTiledFn encode_tiled()
{
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

} // namespace

cudaError_t page_tensor(const uint8_t *pages, const ChunkLaunch &L, CUtensorMap *map)
{
    const EncodeTiledFn enc = encode_tiled();
    if (enc == nullptr)
        return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {kHeadDim, static_cast<cuuint64_t>(L.pm.n_phys) * L.Hkv * kPageTokens};
    const cuuint64_t strides[1] = {kHeadDim};
    const cuuint32_t box[2] = {kHeadDim, kPageTokens}, ones[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(pages), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

} // namespace chunk

namespace {

// Rows of the longest chunk that share a kv head, up to which the kernel for few rows is taken: one of
// its tiles.  (32 users of 4k keys, 4 heads a group: chunks of 8 tokens 100 us against 121 us with the
// large tiles, of 12 tokens 150 us against 123 us; 4 users of 8k: 49 us either way, 57 against 51 us.)
constexpr int64_t kFewRows = 32;

int64_t rows_of(int Hq, int Hkv, int max_q_len) { return static_cast<int64_t>(max_q_len) * (Hq / Hkv); }

} // namespace

size_t chunk_workspace(int, int64_t, int Hq, int Hkv, int max_q_len)
{
    const int64_t rows = rows_of(Hq, Hkv, max_q_len);
    return rows <= kFewRows ? chunk::decode_workspace(static_cast<int>(rows)) : chunk::tiles_workspace();
}

cudaError_t chunk_launch(const ChunkLaunch &launch, cudaStream_t st)
{
    ChunkLaunch L = launch;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const int64_t rows = rows_of(L.Hq, L.Hkv, L.max_q_len);
    return rows <= kFewRows ? chunk::decode_launch(L, static_cast<int>(rows), sms, st) : chunk::tiles_launch(L, sms, st);
}

} // namespace pw
