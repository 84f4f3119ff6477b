// pw_tokens.h -- launch descriptors of the calls on new tokens (pw_qk_norm_rope, pw_append,
// pw_chunk_attn), shared by their entry points (pw_tokens_api.cu) and kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/pw.h"

namespace pw {

// Rows of heads: element (t, h, d) at p[t * st + h * sh + d].
struct RowsIn {
    const uint16_t *p; // bf16 bits
    int64_t st, sh;
    int heads;
    const uint16_t *w; // norm weight, bf16 bits (null: no norm); head h's at w + h * w_stride
    int w_stride;
};

struct RowsOut {
    uint16_t *p;
    int64_t st, sh;
};

// New tokens of a ragged batch: token i of sequence b at row cu[b] + i and position ctx[b] + i.
struct TokenBatch {
    const int32_t *cu, *ctx; // ctx null: 0
    int B;
    int64_t T;
};

struct Rotation {
    const float *table; // [max_pos, rot]: cos, then sin
    int max_pos, rot, interleaved;
};

struct PageMap {
    const int32_t *table;
    int max_pages, n_phys;
};

struct NormRopeLaunch {
    RowsIn q, k;
    RowsOut qo, ko;
    float eps;
    Rotation rope;
    TokenBatch tb;
    int32_t *status;
};

struct AppendLaunch {
    RowsIn k, v;
    float eps, inv_k, inv_v; // 1 / k_scale, 1 / v_scale
    Rotation rope;
    TokenBatch tb;
    PageMap pm;
    uint8_t *K, *V; // E4M3 codes
    int32_t *status;
};

struct ChunkLaunch {
    const uint16_t *Q; // bf16 bits
    int64_t q_st, q_sh;
    const uint8_t *K, *V; // E4M3 codes
    PageMap pm;
    TokenBatch tb;
    int Hq, Hkv, G, window, max_q_len;
    uint32_t g_mul, g_shift; // n / G = (n * g_mul / 2^32 + n) >> g_shift for 0 <= n < 2^31
    uint64_t ctas_mul; // n / CTAs = n * ctas_mul / 2^64 (n below 2^56)
    float score_scale; // sm_scale * k_scale * log2 e: scores to base-2 exponents
    float v_scale;
    uint16_t *O; // bf16 bits
    float *lse;
    void *workspace;
    int32_t *status;
};

cudaError_t norm_rope_launch(const NormRopeLaunch &L, cudaStream_t st);
cudaError_t append_launch(const AppendLaunch &L, cudaStream_t st);
size_t chunk_workspace(int B, int64_t T, int Hq, int Hkv, int max_q_len);
cudaError_t chunk_launch(const ChunkLaunch &L, cudaStream_t st);

} // namespace pw
