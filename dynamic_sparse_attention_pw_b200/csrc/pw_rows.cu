// pw_rows.cu -- pw_qk_norm_rope and pw_append: per-head RMS norm and position rotation of query
// and key rows, and the E4M3 append of keys and values to the paged cache.
//
// A row of 128 bf16 belongs to eight lanes, each with two 16-byte chunks: lane l < rot/16 holds
// the chunks whose elements pair up under the rotation (chunk l and chunk l + rot/16, or for
// neighbouring pairs chunks 2l and 2l + 1), so a pair never crosses lanes, and the lane's cos and
// sin are elements 8l .. 8l + 7 of the table row either way.  The lanes behind take the rest two
// by two.  The norm is three shuffles.
//
// A warp works on heads of one token, four rows at a time.  What they share is formed once: the
// rotation's factors, times the norm weight where all heads have one, so that a row is, per pair,
//   y0 = r (x0 a - x1 b),  y1 = r (x0 c + x1 d),   r = 1 / sqrt(mean(x^2) + eps)
// on packed fp32 pairs.  (A first form that applied weight and rotation row by row was bound by its
// instructions, 71% of the issue slots at 67% of the memory rate.)  How many heads a warp takes is a
// matter of filling the GPU: few tokens, one group of four heads each; many, up to kMost groups.
// A prompt of 16k tokens, 64 + 8 heads (0.6 GB): 106 to 109 us, 5.6 TB/s; sixteen groups a warp 113 us where two
// took 180 us.  Append of two such prompts (8 + 8 heads, 0.2 GB): 49 us (the values go out before the keys'
// factors are formed); its warps have only four groups, and the chain position, page, table row before the
// first store bounds them.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pw_tokens.cuh"

namespace pw {
namespace {

using namespace tokens;

constexpr int kWarps = 4;

__device__ __forceinline__ F2 swap2(F2 v)
{
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(hi, lo);
}

__device__ __forceinline__ void unpack8(const uint4 v, F2 *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pack2(bf16_lo(w[i]), bf16_hi(w[i]));
}

__device__ __forceinline__ uint4 pack8(const F2 *x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(x[i], lo, hi);
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 codes8(const F2 *x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(x[i], lo, hi);
        w[i] = e4m3x2(lo, hi);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The two chunks of lane l of a row.
struct Chunks {
    int c0, c1;
    bool turn;

    __device__ __forceinline__ Chunks(const Rotation &r, int l)
    {
        const int m = r.rot >> 4;
        turn = l < m;
        const bool halves = turn && !r.interleaved;
        c0 = halves ? l : 2 * l;
        c1 = halves ? l + m : 2 * l + 1;
    }
};

// What a lane does to the elements of its chunks, x[0..3] and x[4..7] as pairs.  kInter: neighbours are
// rotated (pair i of both chunks), else pair i of the first with pair i of the second chunk.
template <bool kInter>
struct Turn {
    F2 p[8], q[8];
    bool turn;

    // table row of position pos (not read where the lane's elements are not rotated), weight (null: 1),
    // and a factor for everything
    __device__ __forceinline__ void form(const Rotation &r, const Chunks &ch, int l, int64_t pos, const uint16_t *w, float factor)
    {
        turn = ch.turn;
        F2 g[8];
        const F2 f2 = pack2(factor, factor);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            g[i] = f2;
        if (w != nullptr) {
            unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + ch.c0), g);
            unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + ch.c1), g + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = mul2(g[i], f2);
        }
        if (!turn) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = g[i];
                q[i] = 0ull;
            }
            return;
        }
        F2 cs[4], sn[4];
        const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(r.table + pos * r.rot + 8 * l);
        const ulonglong2 *s = reinterpret_cast<const ulonglong2 *>(r.table + pos * r.rot + (r.rot >> 1) + 8 * l);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const ulonglong2 a = __ldg(c + i), b = __ldg(s + i);
            cs[2 * i] = a.x;
            cs[2 * i + 1] = a.y;
            sn[2 * i] = b.x;
            sn[2 * i + 1] = b.y;
        }
        if (kInter) { // (y0, y1) = (x0, x1) (g0 cos, g1 cos) + (x1, x0) (-g1 sin, g0 sin)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float c0, c1, s0, s1, g0, g1;
                unpack2(cs[i >> 1], c0, c1);
                unpack2(sn[i >> 1], s0, s1);
                unpack2(g[i], g0, g1);
                const float ci = i & 1 ? c1 : c0, si = i & 1 ? s1 : s0;
                p[i] = pack2(g0 * ci, g1 * ci);
                q[i] = pack2(-g1 * si, g0 * si);
            }
        } else { // y0 = x0 g0 cos - x1 g1 sin, y1 = x1 g1 cos + x0 g0 sin
            const F2 minus = pack2(-1.f, -1.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = mul2(g[i], cs[i]);
                p[i + 4] = mul2(g[i + 4], cs[i]);
                q[i] = mul2(mul2(g[i + 4], sn[i]), minus);
                q[i + 4] = mul2(g[i], sn[i]);
            }
        }
    }

    __device__ __forceinline__ void apply(F2 (&x)[8]) const
    {
        F2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = mul2(x[i], p[i]);
        if (turn)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = fma2(kInter ? swap2(x[i]) : x[i ^ 4], q[i], y[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = y[i];
    }
};

// All elements times one factor.
struct Times {
    F2 f;

    __device__ __forceinline__ void apply(F2 (&x)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = mul2(x[i], f);
    }
};

// x /= sqrt(mean(x^2) + eps), the row spread over the eight lanes of a group.
__device__ __forceinline__ void rms_norm(F2 (&x)[8], float eps)
{
    F2 a = 0ull, b = 0ull;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        a = fma2(x[i], x[i], a);
        b = fma2(x[i + 1], x[i + 1], b);
    }
    float a0, a1, b0, b1;
    unpack2(a, a0, a1);
    unpack2(b, b0, b1);
    float s = (a0 + a1) + (b0 + b1);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
    const float r = rsqrtf(s * (1.f / kHeadDim) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = mul2(x[i], pack2(r, r));
}

// x *= weight of one head
__device__ __forceinline__ void weigh(F2 (&x)[8], const uint16_t *w, const Chunks &ch)
{
    F2 g[8];
    unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + ch.c0), g);
    unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + ch.c1), g + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = mul2(x[i], g[i]);
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

// The rows of one token and kind (queries, keys or values) that a warp takes, four at a time, kAhead
// times four on their way.
template <int kAhead>
struct RowStream {
    const uint16_t *row;
    int64_t sh;
    int h1;
    Chunks ch;
    uint4 raw[kAhead][2];

    __device__ __forceinline__ void load(int u, int h)
    {
        raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (h < h1) {
            const uint4 *p = reinterpret_cast<const uint4 *>(row + h * sh);
            raw[u][0] = p[ch.c0];
            raw[u][1] = p[ch.c1];
        }
    }

    __device__ __forceinline__ RowStream(const RowsIn &in, int64_t t, int h0, int h1, const Chunks &ch)
        : row(in.p + t * in.st), sh(in.sh), h1(h1), ch(ch)
    {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            load(u, h0 + 4 * u + ((threadIdx.x & 31) >> 3));
    }

    // store(h, pairs) gets what becomes of a row
    template <class Turned, class Store>
    __device__ __forceinline__ void run(const RowsIn &in, int h0, const Turned &turn, float eps, const Store &store)
    {
        const int group = (threadIdx.x & 31) >> 3;
        const bool per_head = in.w != nullptr && in.w_stride != 0;
#pragma unroll 1
        for (int hb = h0; hb < h1; hb += 4 * kAhead)
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = hb + 4 * u + group;
                if (h - group >= h1)
                    break;
                F2 x[8];
                unpack8(raw[u][0], x);
                unpack8(raw[u][1], x + 4);
                load(u, h + 4 * kAhead);
                if (in.w != nullptr)
                    rms_norm(x, eps);
                if (per_head && h < h1)
                    weigh(x, in.w + h * in.w_stride, ch);
                turn.apply(x);
                if (h < h1)
                    store(h, x);
            }
    }
};

// Blocks are kWarps tokens by one stretch of `heads` heads of one kind.
template <bool kInter>
__global__ void __launch_bounds__(32 * kWarps) k_norm_rope(const NormRopeLaunch L, int heads, int q_parts)
{
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= L.tb.T)
        return;
    const bool isq = static_cast<int>(blockIdx.y) < q_parts;
    const RowsIn &in = isq ? L.q : L.k;
    const RowsOut &out = isq ? L.qo : L.ko;
    const int h0 = (static_cast<int>(blockIdx.y) - (isq ? 0 : q_parts)) * heads, h1 = min(h0 + heads, in.heads);
    Chunks ch(L.rope, l);
    RowStream<4> rows(in, t, h0, h1, ch); // on its way while the position is found
    int b;
    int64_t pos;
    if (!place(L.tb, t, lane, b, pos))
        return;
    if (L.rope.rot > 0 && (pos < 0 || pos >= L.rope.max_pos)) { // recorded and not rotated
        set_status(L.status, PW_ERR_INVALID_ARG);
        ch.turn = false;
    }
    Turn<kInter> turn;
    turn.form(L.rope, ch, l, pos, in.w_stride == 0 ? in.w : nullptr, 1.f);
    uint16_t *const row = out.p + t * out.st;
    rows.run(in, h0, turn, L.eps, [&](int h, const F2 (&x)[8]) {
        uint4 *p = reinterpret_cast<uint4 *>(row + h * out.sh);
        p[ch.c0] = pack8(x);
        p[ch.c1] = pack8(x + 4);
    });
}

// Blocks are kWarps tokens by one stretch of `heads` heads, keys and values.
template <bool kInter>
__global__ void __launch_bounds__(32 * kWarps) k_append(const AppendLaunch L, int heads)
{
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= L.tb.T)
        return;
    const int Hkv = L.k.heads, h0 = static_cast<int>(blockIdx.y) * heads, h1 = min(h0 + heads, Hkv);
    const Chunks ck(L.rope, l), cv(Rotation{nullptr, 0, 0, 0}, l);
    RowStream<2> values(L.v, t, h0, h1, cv), keys(L.k, t, h0, h1, ck); // on their way while the position is found
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
    const size_t row = (static_cast<size_t>(phys) * Hkv * kPageTokens + (pos & 63)) * kHeadDim;
    values.run(L.v, h0, Times{pack2(L.inv_v, L.inv_v)}, 0.f, [&](int h, const F2 (&x)[8]) {
        uint2 *p = reinterpret_cast<uint2 *>(L.V + row + static_cast<size_t>(h) * (kPageTokens * kHeadDim));
        const uint2 a = codes8(x), c = codes8(x + 4); // neighbouring chunks
        *reinterpret_cast<uint4 *>(p + cv.c0) = make_uint4(a.x, a.y, c.x, c.y);
    });
    Turn<kInter> turn; // behind the values, which need no table row
    turn.form(L.rope, ck, l, pos, L.k.w_stride == 0 ? L.k.w : nullptr, L.inv_k);
    keys.run(L.k, h0, turn, L.eps, [&](int h, const F2 (&x)[8]) {
        uint2 *p = reinterpret_cast<uint2 *>(L.K + row + static_cast<size_t>(h) * (kPageTokens * kHeadDim));
        p[ck.c0] = codes8(x);
        p[ck.c1] = codes8(x + 4);
    });
}

// Heads a warp takes, a multiple of four: as many as leave the GPU kFill warps an SM, at most kMost groups.
int heads_of_warp(int64_t T, int H)
{
    constexpr int kFill = 32, kMost = 16, kSms = 148;
    const int64_t groups = T * ((H + 3) / 4) / (kFill * kSms);
    return 4 * static_cast<int>(std::min<int64_t>(std::max<int64_t>(groups, 1), kMost));
}

unsigned blocks_for(int64_t T) { return static_cast<unsigned>((T + kWarps - 1) / kWarps); }

} // namespace

cudaError_t norm_rope_launch(const NormRopeLaunch &L, cudaStream_t st)
{
    const int heads = heads_of_warp(L.tb.T, L.q.heads + L.k.heads);
    const int q = (L.q.heads + heads - 1) / heads, k = (L.k.heads + heads - 1) / heads;
    const dim3 grid(blocks_for(L.tb.T), q + k);
    if (L.rope.interleaved)
        k_norm_rope<true><<<grid, 32 * kWarps, 0, st>>>(L, heads, q);
    else
        k_norm_rope<false><<<grid, 32 * kWarps, 0, st>>>(L, heads, q);
    return cudaGetLastError();
}

cudaError_t append_launch(const AppendLaunch &L, cudaStream_t st)
{
    const int heads = heads_of_warp(L.tb.T, L.k.heads);
    const dim3 grid(blocks_for(L.tb.T), (L.k.heads + heads - 1) / heads);
    if (L.rope.interleaved)
        k_append<true><<<grid, 32 * kWarps, 0, st>>>(L, heads);
    else
        k_append<false><<<grid, 32 * kWarps, 0, st>>>(L, heads);
    return cudaGetLastError();
}

} // namespace pw
