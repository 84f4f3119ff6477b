// pw_rows.cu -- pw_qk_norm_rope and pw_append: per-head RMS norm and position rotation of query
// and key rows, and the E4M3 append of keys and values to the paged cache.
//
// A row of 128 bf16 belongs to eight lanes, each with two 16-byte chunks: lane l < rot/16 holds
// the chunks whose elements pair up under the rotation (chunk l and chunk l + rot/16, or for
// neighbouring pairs chunks 2l and 2l + 1), so a pair never crosses lanes, and the lane's cos and
// sin are elements 8l .. 8l + 7 of the table row either way.  The lanes behind take the rest two
// by two.  The norm is three shuffles.  A warp works on one token: four rows at a time, U times,
// with the token's table values in registers for all of them.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pw_tokens.cuh"

namespace pw {
namespace {

using namespace tokens;

constexpr int kWarps = 8;

__device__ __forceinline__ void unpack8(const uint4 v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float *x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 codes8(const float *x, float inv_scale)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = e4m3x2(x[2 * i] * inv_scale, x[2 * i + 1] * inv_scale);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The two chunks of lane l of a row and the rotation of its 8 pairs.
struct Pairs {
    int c0, c1;
    bool turn;
    float cs[8], sn[8];

    __device__ __forceinline__ Pairs(const Rotation &r, int l)
    {
        const int m = r.rot >> 4;
        turn = l < m;
        const bool halves = turn && !r.interleaved;
        c0 = halves ? l : 2 * l;
        c1 = halves ? l + m : 2 * l + 1;
    }

    // cos and sin of position pos; a position outside the table is recorded and not rotated
    __device__ __forceinline__ void load(const Rotation &r, int l, int64_t pos, int32_t *status)
    {
        if (r.rot > 0 && (pos < 0 || pos >= r.max_pos)) {
            set_status(status, PW_ERR_INVALID_ARG);
            turn = false;
        }
        if (!turn)
            return;
        const float4 *p = reinterpret_cast<const float4 *>(r.table + pos * r.rot + 8 * l);
        const float4 *q = reinterpret_cast<const float4 *>(r.table + pos * r.rot + (r.rot >> 1) + 8 * l);
        *reinterpret_cast<float4 *>(cs) = __ldg(p);
        *reinterpret_cast<float4 *>(cs + 4) = __ldg(p + 1);
        *reinterpret_cast<float4 *>(sn) = __ldg(q);
        *reinterpret_cast<float4 *>(sn + 4) = __ldg(q + 1);
    }

    __device__ __forceinline__ void rotate(const Rotation &r, float (&x)[16]) const
    {
        if (!turn)
            return;
        if (r.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = u * cs[i] - v * sn[i];
                x[2 * i + 1] = u * sn[i] + v * cs[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = x[i], v = x[8 + i];
                x[i] = u * cs[i] - v * sn[i];
                x[8 + i] = u * sn[i] + v * cs[i];
            }
        }
    }
};

// x *= weight / sqrt(mean(x^2) + eps), the row spread over the eight lanes of a group.
__device__ __forceinline__ void rms_norm(float (&x)[16], const uint16_t *w, const Pairs &pr, float eps)
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        s = fmaf(x[i], x[i], s);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
    if (w == nullptr)
        return;
    const float r = rsqrtf(s * (1.f / kHeadDim) + eps);
    float g[16];
    unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + pr.c0), g);
    unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + pr.c1), g + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        x[i] *= r * g[i];
}

// Position of row t, or -1 behind the last sequence; the whole warp calls it.
__device__ __forceinline__ bool place(const TokenBatch &tb, int64_t t, int lane, int &b, int64_t &pos)
{
    b = find_sequence(tb, t, lane);
    if (b >= tb.B)
        return false;
    const int64_t i = t - __ldg(tb.cu + b);
    pos = i + (tb.ctx != nullptr ? __ldg(tb.ctx + b) : 0);
    return i >= 0;
}

template <int U>
__global__ void __launch_bounds__(32 * kWarps) k_norm_rope(const NormRopeLaunch L)
{
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int H = L.q.heads + L.k.heads, items = (H + 4 * U - 1) / (4 * U);
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t = w / items;
    if (t >= L.tb.T)
        return;
    const int h0 = static_cast<int>(w - t * items) * 4 * U + (lane >> 3);
    Pairs pr(L.rope, l);
    uint4 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + 4 * u;
        raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (h < H) {
            const bool isq = h < L.q.heads;
            const RowsIn &r = isq ? L.q : L.k;
            const uint4 *p = reinterpret_cast<const uint4 *>(r.p + t * r.st + (isq ? h : h - L.q.heads) * r.sh);
            raw[u][0] = p[pr.c0];
            raw[u][1] = p[pr.c1];
        }
    }
    int b;
    int64_t pos;
    if (!place(L.tb, t, lane, b, pos))
        return;
    pr.load(L.rope, l, pos, L.status);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + 4 * u;
        const bool isq = h < L.q.heads;
        const RowsIn &r = isq ? L.q : L.k;
        const RowsOut &o = isq ? L.qo : L.ko;
        const int hh = isq ? h : h - L.q.heads;
        float x[16];
        unpack8(raw[u][0], x);
        unpack8(raw[u][1], x + 8);
        rms_norm(x, h < H && r.w != nullptr ? r.w + hh * r.w_stride : nullptr, pr, L.eps);
        pr.rotate(L.rope, x);
        if (h < H) {
            uint4 *p = reinterpret_cast<uint4 *>(o.p + t * o.st + hh * o.sh);
            p[pr.c0] = pack8(x);
            p[pr.c1] = pack8(x + 8);
        }
    }
}

template <int U>
__global__ void __launch_bounds__(32 * kWarps) k_append(const AppendLaunch L)
{
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int Hkv = L.k.heads, H = 2 * Hkv, items = (H + 4 * U - 1) / (4 * U);
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t = w / items;
    if (t >= L.tb.T)
        return;
    const int h0 = static_cast<int>(w - t * items) * 4 * U + (lane >> 3);
    Pairs pr(L.rope, l);
    uint4 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + 4 * u;
        raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (h < H) {
            const RowsIn &r = h < Hkv ? L.k : L.v;
            const uint4 *p = reinterpret_cast<const uint4 *>(r.p + t * r.st + (h < Hkv ? h : h - Hkv) * r.sh);
            raw[u][0] = p[pr.c0];
            raw[u][1] = p[pr.c1];
        }
    }
    int b;
    int64_t pos;
    if (!place(L.tb, t, lane, b, pos))
        return;
    const int64_t page = pos >> 6;
    int phys = -1;
    if (pos >= 0 && page < L.pm.max_pages)
        phys = __ldg(L.pm.table + static_cast<int64_t>(b) * L.pm.max_pages + page);
    if (phys < 0 || phys >= L.pm.n_phys || (L.rope.rot > 0 && pos >= L.rope.max_pos)) {
        set_status(L.status, PW_ERR_INVALID_ARG);
        return;
    }
    pr.load(L.rope, l, pos, L.status);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + 4 * u;
        const bool isk = h < Hkv;
        const int hh = isk ? h : h - Hkv;
        float x[16];
        unpack8(raw[u][0], x);
        unpack8(raw[u][1], x + 8);
        rms_norm(x, isk && L.k.w != nullptr ? L.k.w + hh * L.k.w_stride : nullptr, pr, L.eps);
        if (isk)
            pr.rotate(L.rope, x);
        if (h < H) {
            uint2 *p = reinterpret_cast<uint2 *>((isk ? L.K : L.V) +
                                                 ((static_cast<size_t>(phys) * Hkv + hh) * kPageTokens + (pos & 63)) * kHeadDim);
            const float inv = isk ? L.inv_k : L.inv_v;
            p[pr.c0] = codes8(x, inv);
            p[pr.c1] = codes8(x + 8, inv);
        }
    }
}

template <int U>
unsigned blocks_for(int64_t T, int H)
{
    const int64_t items = (H + 4 * U - 1) / (4 * U);
    return static_cast<unsigned>((T * items + kWarps - 1) / kWarps);
}

} // namespace

cudaError_t norm_rope_launch(const NormRopeLaunch &L, cudaStream_t st)
{
    const int H = L.q.heads + L.k.heads;
    k_norm_rope<1><<<blocks_for<1>(L.tb.T, H), 32 * kWarps, 0, st>>>(L);
    return cudaGetLastError();
}

cudaError_t append_launch(const AppendLaunch &L, cudaStream_t st)
{
    k_append<1><<<blocks_for<1>(L.tb.T, 2 * L.k.heads), 32 * kWarps, 0, st>>>(L);
    return cudaGetLastError();
}

} // namespace pw
