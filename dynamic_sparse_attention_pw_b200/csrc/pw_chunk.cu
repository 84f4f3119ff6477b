// pw_chunk.cu -- pw_chunk_attn: causal attention of new tokens over the paged E4M3 cache.
//
// One warp per (row, query head): 32 keys at a time, lane d4 holds four dimensions of q, k and v;
// the scores of the 32 keys go to one lane each, the softmax is online in fp32, base 2.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pw_chunk.cuh"

namespace pw {
namespace {

using namespace tokens;
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t x, float (&f)[4])
{
    uint32_t a, b;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}\n"
        : "=r"(a), "=r"(b) : "r"(x));
    const __half2 p = *reinterpret_cast<const __half2 *>(&a), q = *reinterpret_cast<const __half2 *>(&b);
    f[0] = __low2float(p);
    f[1] = __high2float(p);
    f[2] = __low2float(q);
    f[3] = __high2float(q);
}

__global__ void __launch_bounds__(256) k_chunk_rows(const ChunkLaunch L)
{
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = w / L.Hq;
    const int hq = static_cast<int>(w - t * L.Hq), h = hq / L.G;
    if (t >= L.tb.T)
        return;
    const int b = find_sequence(L.tb, t, lane);
    if (b >= L.tb.B)
        return;
    const int64_t i = t - L.tb.cu[b];
    if (i < 0)
        return;
    int64_t pos = i + (L.tb.ctx != nullptr ? L.tb.ctx[b] : 0);
    if (pos < 0 || pos >= static_cast<int64_t>(L.pm.max_pages) * 64) {
        set_status(L.status, PW_ERR_INVALID_ARG);
        pos = min(max(pos, static_cast<int64_t>(0)), static_cast<int64_t>(L.pm.max_pages) * 64 - 1);
    }
    const int64_t first = L.window > 0 ? max(pos - L.window + 1, static_cast<int64_t>(0)) : 0;
    const uint2 qr = *reinterpret_cast<const uint2 *>(L.Q + t * L.q_st + hq * L.q_sh + 4 * lane);
    const float c = L.score_scale;
    const float q[4] = {bf16_lo(qr.x) * c, bf16_hi(qr.x) * c, bf16_lo(qr.y) * c, bf16_hi(qr.y) * c};
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = first & ~31ll; k0 <= pos; k0 += 32) {
        int phys = L.pm.table[static_cast<int64_t>(b) * L.pm.max_pages + (k0 >> 6)];
        if (phys < 0 || phys >= L.pm.n_phys) {
            set_status(L.status, PW_ERR_INVALID_ARG);
            phys = 0;
        }
        const size_t row = (static_cast<size_t>(phys) * L.Hkv + h) * 64 + (k0 & 63);
        float s = -INFINITY;
#pragma unroll 4
        for (int j = 0; j < 32; ++j) {
            float k[4];
            e4m3x4_to_f32(reinterpret_cast<const uint32_t *>(L.K + (row + j) * 128)[lane], k);
            float d = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
            for (int x = 16; x > 0; x >>= 1)
                d += __shfl_xor_sync(kFull, d, x);
            if (lane == j && k0 + j >= first && k0 + j <= pos)
                s = d;
        }
        float mx = s;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, x));
        mx = fmaxf(mx, m);
        const float a = exp2f(m - mx), p = exp2f(s - mx);
        m = mx;
        l = l * a + p;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] *= a;
#pragma unroll 4
        for (int j = 0; j < 32; ++j) {
            const float pj = __shfl_sync(kFull, p, j);
            if (k0 + j < first || k0 + j > pos)
                continue;
            float v[4];
            e4m3x4_to_f32(reinterpret_cast<const uint32_t *>(L.V + (row + j) * 128)[lane], v);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fmaf(pj, v[e], o[e]);
        }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
        l += __shfl_xor_sync(kFull, l, x);
    const float inv = L.v_scale / l;
    const __nv_bfloat162 r0 = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), r1 = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2 *>(L.O + (t * L.Hq + hq) * 128 + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&r0), *reinterpret_cast<const uint32_t *>(&r1));
    if (L.lse != nullptr && lane == 0)
        L.lse[t * L.Hq + hq] = (m + log2f(l)) * 0.6931471805599453f;
}

} // namespace

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

size_t chunk_workspace(int, int64_t, int Hq, int Hkv, int max_q_len)
{
    return chunk::decode_workspace(static_cast<int>(min(static_cast<int64_t>(max_q_len) * (Hq / Hkv), static_cast<int64_t>(1) << 20)));
}

cudaError_t chunk_launch(const ChunkLaunch &L, cudaStream_t st)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const int64_t rows = static_cast<int64_t>(L.max_q_len) * L.G;
    if (rows <= 64)
        return chunk::decode_launch(L, static_cast<int>(rows), min(sms, chunk::kMaxCtas), st);
    k_chunk_rows<<<static_cast<unsigned>((L.tb.T * L.Hq + 7) / 8), 256, 0, st>>>(L);
    return cudaGetLastError();
}

} // namespace pw
