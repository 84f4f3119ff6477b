// pw_tokens_api.cu -- entry points of the calls on new tokens declared in include/pw.h
// (pw_qk_norm_rope, pw_append, pw_chunk_attn): argument checks on the host, then the launches.
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "pw_internal.h"
#include "pw_tokens.h"

namespace {

using namespace pw;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool finite_positive(float x) { return std::isfinite(x) && x > 0.f; }

// Rows of heads as an input: any strides that keep every row on a 16-byte boundary.
pw_status check_in(const void *p, int64_t st, int64_t sh, int heads)
{
    if (heads == 0)
        return PW_OK;
    if (!p || !aligned16(p) || ((st | sh) & 7))
        return PW_ERR_INVALID_ARG;
    return PW_OK;
}

// As an output the rows must not overlap either: tokens outermost or heads outermost.
pw_status check_out(const void *p, int64_t st, int64_t sh, int heads, int64_t T)
{
    if (heads == 0)
        return PW_OK;
    const pw_status s = check_in(p, st, sh, heads);
    if (s != PW_OK)
        return s;
    const bool by_token = (heads == 1 || sh >= kHeadDim) && (T == 1 || st >= (heads - 1) * sh + kHeadDim);
    const bool by_head = (T == 1 || st >= kHeadDim) && (heads == 1 || sh >= (T - 1) * st + kHeadDim);
    return by_token || by_head ? PW_OK : PW_ERR_INVALID_ARG;
}

pw_status check_norm(const void *w, int stride)
{
    return !w || (aligned16(w) && (stride == 0 || stride == kHeadDim)) ? PW_OK : PW_ERR_INVALID_ARG;
}

pw_status check_rope(const float *rope, int max_pos, int &rot)
{
    if (!rope || rot == 0) {
        rot = 0;
        return PW_OK;
    }
    if (rot < 0 || max_pos < 1 || !aligned16(rope))
        return PW_ERR_INVALID_ARG;
    return rot % 16 == 0 && rot <= kHeadDim ? PW_OK : PW_ERR_UNSUPPORTED;
}

pw_status check_batch(const int32_t *cu, int B, int64_t T)
{
    if (!cu || B < 1 || T < 0)
        return PW_ERR_INVALID_ARG;
    return T < (int64_t(1) << 31) ? PW_OK : PW_ERR_UNSUPPORTED;
}

// The second dimension of the grid counts heads by four.
bool grid_fits(int64_t heads) { return heads <= 4 * 32767; }

#define PW_TRY(x)                                                                                  \
    do {                                                                                           \
        const pw_status pw_try_ = (x);                                                             \
        if (pw_try_ != PW_OK)                                                                      \
            return pw_try_;                                                                        \
    } while (0)

} // namespace

extern "C" {

pw_status pw_qk_norm_rope(const void *Q, int64_t q_stride_t, int64_t q_stride_h, int Hq,
                          const void *K, int64_t k_stride_t, int64_t k_stride_h, int Hk,
                          const void *q_weight, int q_weight_stride, const void *k_weight,
                          int k_weight_stride, float eps, const float *rope, int max_pos,
                          int rot_dim, int interleaved, const int32_t *cu_seqlens,
                          const int32_t *ctx_lens, int B, int64_t T, void *Q_out,
                          int64_t qo_stride_t, int64_t qo_stride_h, void *K_out,
                          int64_t ko_stride_t, int64_t ko_stride_h, int32_t *dev_status,
                          void *stream)
{
    if (Hq < 0 || Hk < 0 || Hq + static_cast<int64_t>(Hk) < 1 || !(eps >= 0.f) || !std::isfinite(eps))
        return PW_ERR_INVALID_ARG;
    PW_TRY(check_batch(cu_seqlens, B, T));
    PW_TRY(check_norm(q_weight, q_weight_stride));
    PW_TRY(check_norm(k_weight, k_weight_stride));
    PW_TRY(check_rope(rope, max_pos, rot_dim));
    if (T == 0)
        return PW_OK;
    if (!grid_fits(Hq + static_cast<int64_t>(Hk)))
        return PW_ERR_UNSUPPORTED;
    PW_TRY(check_in(Q, q_stride_t, q_stride_h, Hq));
    PW_TRY(check_in(K, k_stride_t, k_stride_h, Hk));
    PW_TRY(check_out(Q_out, qo_stride_t, qo_stride_h, Hq, T));
    PW_TRY(check_out(K_out, ko_stride_t, ko_stride_h, Hk, T));
    NormRopeLaunch L{};
    L.q = {static_cast<const uint16_t *>(Q), q_stride_t, q_stride_h, Hq,
           static_cast<const uint16_t *>(q_weight), q_weight_stride};
    L.k = {static_cast<const uint16_t *>(K), k_stride_t, k_stride_h, Hk,
           static_cast<const uint16_t *>(k_weight), k_weight_stride};
    L.qo = {static_cast<uint16_t *>(Q_out), qo_stride_t, qo_stride_h};
    L.ko = {static_cast<uint16_t *>(K_out), ko_stride_t, ko_stride_h};
    L.eps = eps;
    L.rope = {rope, max_pos, rot_dim, interleaved != 0};
    L.tb = {cu_seqlens, ctx_lens, B, T};
    L.status = dev_status;
    return norm_rope_launch(L, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PW_OK : PW_ERR_CUDA;
}

pw_status pw_append(const void *K, int64_t k_stride_t, int64_t k_stride_h, const void *V,
                    int64_t v_stride_t, int64_t v_stride_h, int Hkv, const void *k_weight,
                    int k_weight_stride, float eps, const float *rope, int max_pos, int rot_dim,
                    int interleaved, const int32_t *cu_seqlens, const int32_t *ctx_lens, int B,
                    int64_t T, const int32_t *page_table, int max_pages, int n_phys,
                    float k_scale, float v_scale, void *K_pages, void *V_pages,
                    int32_t *dev_status, void *stream)
{
    if (Hkv < 1 || max_pages < 0 || n_phys < 0 || !(eps >= 0.f) || !std::isfinite(eps) ||
        !finite_positive(k_scale) || !finite_positive(v_scale) || !std::isfinite(1.f / k_scale) ||
        !std::isfinite(1.f / v_scale))
        return PW_ERR_INVALID_ARG;
    PW_TRY(check_batch(cu_seqlens, B, T));
    PW_TRY(check_norm(k_weight, k_weight_stride));
    PW_TRY(check_rope(rope, max_pos, rot_dim));
    if (T == 0)
        return PW_OK;
    if (!grid_fits(2 * static_cast<int64_t>(Hkv)))
        return PW_ERR_UNSUPPORTED;
    PW_TRY(check_in(K, k_stride_t, k_stride_h, Hkv));
    PW_TRY(check_in(V, v_stride_t, v_stride_h, Hkv));
    if (!page_table || !K_pages || !V_pages || !aligned16(K_pages) || !aligned16(V_pages))
        return PW_ERR_INVALID_ARG;
    AppendLaunch L{};
    L.k = {static_cast<const uint16_t *>(K), k_stride_t, k_stride_h, Hkv,
           static_cast<const uint16_t *>(k_weight), k_weight_stride};
    L.v = {static_cast<const uint16_t *>(V), v_stride_t, v_stride_h, Hkv, nullptr, 0};
    L.eps = eps;
    L.inv_k = 1.f / k_scale;
    L.inv_v = 1.f / v_scale;
    L.rope = {rope, max_pos, rot_dim, interleaved != 0};
    L.tb = {cu_seqlens, ctx_lens, B, T};
    L.pm = {page_table, max_pages, n_phys};
    L.K = static_cast<uint8_t *>(K_pages);
    L.V = static_cast<uint8_t *>(V_pages);
    L.status = dev_status;
    return append_launch(L, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PW_OK : PW_ERR_CUDA;
}

pw_status pw_chunk_workspace_size(int B, int64_t T, int Hq, int Hkv, int max_q_len,
                                  size_t *workspace_bytes)
{
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || max_q_len < 1 || !workspace_bytes)
        return PW_ERR_INVALID_ARG;
    if (Hq % Hkv != 0)
        return PW_ERR_UNSUPPORTED;
    *workspace_bytes = chunk_workspace(B, T, Hq, Hkv, max_q_len);
    return PW_OK;
}

pw_status pw_chunk_attn(const void *Q, int64_t q_stride_t, int64_t q_stride_h, int Hq,
                        const void *K_pages, const void *V_pages, int Hkv,
                        const int32_t *page_table, int max_pages, int n_phys,
                        const int32_t *cu_seqlens, const int32_t *ctx_lens, int B, int64_t T,
                        int max_q_len, int window, float k_scale, float v_scale, float sm_scale,
                        void *O, float *lse, void *workspace, size_t workspace_bytes,
                        int32_t *dev_status, void *stream)
{
    size_t need = 0;
    PW_TRY(pw_chunk_workspace_size(B, T, Hq, Hkv, max_q_len, &need));
    PW_TRY(check_batch(cu_seqlens, B, T));
    if (max_pages < 1 || n_phys < 1 || window < 0)
        return PW_ERR_INVALID_ARG;
    const double scale = static_cast<double>(sm_scale) * k_scale * 1.4426950408889634;
    if (!finite_positive(sm_scale) || !finite_positive(k_scale) || !finite_positive(v_scale) ||
        !finite_positive(static_cast<float>(scale)))
        return PW_ERR_INVALID_ARG;
    if (max_pages > (1 << 24) || static_cast<int64_t>(n_phys) * Hkv * kPageTokens > 0x7FFFFFFFll)
        return PW_ERR_UNSUPPORTED; // positions, and cache rows, are addressed with 32 bits
    if (T == 0)
        return PW_OK;
    if (T * static_cast<int64_t>(Hq) > 0x7FFFF000ll)
        return PW_ERR_UNSUPPORTED; // rows are counted with 32 bits
    PW_TRY(check_in(Q, q_stride_t, q_stride_h, Hq));
    if (!K_pages || !V_pages || !page_table || !O || !aligned16(K_pages) || !aligned16(V_pages) || !aligned16(O))
        return PW_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need)
        return PW_ERR_CAPACITY;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return PW_ERR_INVALID_ARG;
    ChunkLaunch L{};
    L.Q = static_cast<const uint16_t *>(Q);
    L.q_st = q_stride_t;
    L.q_sh = q_stride_h;
    L.K = static_cast<const uint8_t *>(K_pages);
    L.V = static_cast<const uint8_t *>(V_pages);
    L.pm = {page_table, max_pages, n_phys};
    L.tb = {cu_seqlens, ctx_lens, B, T};
    L.Hq = Hq;
    L.Hkv = Hkv;
    L.G = Hq / Hkv;
    while ((1ll << L.g_shift) < L.G)
        ++L.g_shift;
    L.g_mul = static_cast<uint32_t>((((1ull << L.g_shift) - L.G) << 32) / L.G + 1);
    L.window = window;
    L.max_q_len = max_q_len;
    L.score_scale = static_cast<float>(scale);
    L.v_scale = v_scale;
    L.O = static_cast<uint16_t *>(O);
    L.lse = lse;
    L.workspace = workspace;
    L.status = dev_status;
    return chunk_launch(L, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PW_OK : PW_ERR_CUDA;
}

} // extern "C"
