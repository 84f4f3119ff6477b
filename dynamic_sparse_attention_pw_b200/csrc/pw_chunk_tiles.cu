// pw_chunk_tiles.cu -- pw_chunk_attn for many rows: chunks of a prompt.
//
// A tile is 256 rows, two halves of 128, against blocks of 128 keys.  Per half and block
//   S = q1 K^T + q2 K^T   (M = 128 rows, N = 128 keys; E4M3 K as stored, the query's E4M3 and E5M2 parts)
//   O += P V              (M = 128 rows, N = 128 dims, K = 128 keys; f16: P from TMEM, V converted)
// The 8-bit products of the two query parts take as long as one bf16 product would and spare the
// conversion of K; V is converted (exactly) to f16 once for both halves.  The halves alternate: while
// one is in the softmax, the tensor cores work for the other.  The softmax is one thread a row: no
// reduction crosses threads.
//
// A row's running maximum is a reference, a whole number, that moves when a score of a chunk of 32
// keys exceeds it by more than 2^15 (f16 ends at 2^16); what the row has so far, the weights of the
// block's earlier chunks among it, is then scaled by a power of two.  It lies less than 1 above the row's largest
// score when it moves, so that the largest weight is more than 1/2 and a weight below f16's normal range is off by
// at most 2^-24 of it.  (Whole numbers below the score would halve that, and measured 203 us against 196 on
// ragged chunks.)
//
// Weights enter P V as one f16, 2^-11 of themselves off at most, where pw_attn carries a second f16 with the rest:
// from the 64-bit result, outputs differ by 1.68e-3 rel-L2, of which bf16's rounding alone makes 1.66e-3
// (rounded to bf16, the two differ by up to 9.7e-4).  The second products would take the tensor cores from
// 2400 to 3540 of a block's 3500 cycles: 2.41 ms where 1.89 are taken (2048 tokens at 32k).
//
//   warps 0-3    softmax, first half; the end of its rows
//   warps 4-7    softmax, second half
//   warps 8-11   the next tile's queries; V to f16
//   warp 12      load: page ids, copies of K and V, job records
//   warp 13      the products
// What bounds it: the chain of a half's block -- softmax 1650 to 2050 cycles, wake-up 350, P V 570, S 600,
// S back to the softmax 240 -- of which the other half's hides most: a block of 256 rows takes 3500
// cycles, the tensor cores' share of it 2400.  2048 tokens at 32k (2.13 TFLOP): 1.88 to 1.93 ms a call
// in a row, under the power limit (1.64 ms with a pause and a flushed L2 before each).  Tried and slower: a product warp for each half (the halves
// fall into step: 2.14 ms against 1.73), steps of 64 keys with S a step ahead (M = 128, N = 64 products
// take as long as N = 128: 2.48), two threads a row (1.79), part of the exponentials on the
// multiply-add units (a quarter of them 1.86), waits that spin (1.79).
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pw_chunk.cuh"

namespace pw {
namespace chunk {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 256;
constexpr int kHalf = 128;
constexpr int kJobs = 4;
constexpr int kNK = 3, kNV = 2; // K and V stages
constexpr float kRaise = 15.f;  // a row's reference moves when a score exceeds it by more (base 2); f16 ends at 2^16

struct __align__(1024) TileSmem {
    uint8_t q[2][2][kHalf * 128];   // [half][part][row][dim] E4M3, E5M2
    uint8_t k[kNK][kBlock * 128];   // E4M3, swizzled by the copy
    uint8_t v[kNV][kBlock * 128];   // E4M3 as stored
    uint8_t v16[2][2][kBlock * 128]; // [block % 2][dims 0-63, 64-127][key][dim] f16, swizzled
    float c[2][2][kHalf];           // [half][its tile % 2]: factor of a row's scores
    // [half][its tile % 3]: NaN for a row that sees a value taken out as NaN, else 0.  Any of the V warps
    // marks any row, without waiting for the others, so the thread that reads a mark clears it.  Three,
    // because a tile's are read at its end, when the values of the next two tiles may be marked already; those
    // of the third come behind products that its softmax warps let go after that end.
    float bad[2][3][kHalf];
    Job job[kJobs];
    uint64_t job_full[kJobs], job_empty[kJobs];
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kNK], k_empty[kNK], v_full[kNV], v_empty[kNV];
    uint64_t v16_full[2], v16_empty[2];
    uint64_t s_full[2], p_most[2], p_full[2], o_full[2], o_free[2]; // p_most: all weights of a block but the last 32 keys'
    uint64_t drain;
    uint32_t k_issued, v_issued; // blocks whose copies were issued
    uint32_t tmem;
    int32_t abort_flag;
};
static_assert(sizeof(TileSmem) + 1024 <= 227 * 1024, "shared-memory layout too large");

__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ int halves(const Job &j) { return j.rows > kHalf ? 2 : 1; }

// Sixteen E4M3 codes to f16.
__device__ __forceinline__ void e4m3x16_to_f16(const uint4 x, uint4 &h0, uint4 &h1)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}\n"
            : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
            : "r"(w[i]));
    h0 = make_uint4(h[0], h[1], h[2], h[3]);
    h1 = make_uint4(h[4], h[5], h[6], h[7]);
}

// 32 bytes, a whole sector: rows of one thread each, so a warp's stores touch 32 places.
__device__ __forceinline__ void store32(void *p, const uint32_t *r)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
                 "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ float max32(const uint32_t (&x)[32])
{
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; e += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t[i] = fmaxf(t[i], fmaxf(__uint_as_float(x[e + 2 * i]), __uint_as_float(x[e + 2 * i + 1])));
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// A thread's row times alpha, a power of two: no pieces of 16 dims of its accumulator, and np pieces
// of 32 weights.  The products issued so far are complete: the scores at hand were issued after them.
static __device__ __noinline__ void rescale(uint32_t o_addr, int no, uint32_t p_addr, int np, float alpha)
{
    tmem_st_wait();
#pragma unroll 1
    for (int i = 0; i < no + np; ++i) {
        const uint32_t at = i < no ? o_addr + 16 * i : p_addr + 16 * (i - no);
        uint32_t x[16];
        tmem_ld16(at, x);
        tmem_ld_wait16(x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[e]));
            const __half2 w = __floats2half2_rn(f.x * alpha, f.y * alpha); // alpha itself may lie below f16's range
            x[e] = i < no ? __float_as_uint(__uint_as_float(x[e]) * alpha) : *reinterpret_cast<const uint32_t *>(&w);
        }
        tmem_st16(at, x);
    }
    tmem_st_wait();
}

// Takes the NaN out of the values of the block at b0 (the pieces that thread t converts); the rows of the
// tile that see such a key get one.  Rare, and so not inlined.
static __device__ __noinline__ void take_nan(uint8_t *v, int t, int b0, int lo, int hi, const Shape shape, int ctx, int row, int rows, float *bad0,
                                             float *bad1)
{
#pragma unroll 1
    for (int q = t; q < kBlock * 8; q += 128) {
        const int kp = b0 + (q >> 3);
        if (kp < lo || kp >= hi)
            continue; // any bytes
        uint4 *const at = reinterpret_cast<uint4 *>(v + q * 16);
        uint4 x = *at;
        if (!drop_nan(x))
            continue;
        *at = x;
#pragma unroll 1
        for (int r = 0; r < rows; ++r) {
            const int pos = shape.position(ctx, shape.token(row + r));
            if (pos >= kp && (shape.window == 0 || pos - kp < shape.window))
                (r < kHalf ? bad0 : bad1)[r & (kHalf - 1)] = __int_as_float(0x7FC00000);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_tiles(const ChunkLaunch L, const __grid_constant__ CUtensorMap map_k)
{
    constexpr uint32_t kIdescS = idesc_e4m3_f32(128, 128), kIdescRest = kIdescS | (1u << 7); // A: E5M2
    constexpr uint32_t kIdescO = idesc_f16_f32(128, 128, false, true);
    constexpr uint32_t kColS = 128, kColO = 256; // S / P of the halves at columns 0 and 128, O at 256 and 384
    extern __shared__ uint8_t smem_raw[];
    TileSmem &sm = *reinterpret_cast<TileSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;

    for (int i = tid; i < 2 * 3 * kHalf; i += kThreads)
        (&sm.bad[0][0][0])[i] = 0.f;
    if (tid == 0) {
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&sm.job_full[i], 1);
            mbar_init(&sm.job_empty[i], 8 + 4 + 1); // softmax, query and product warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 4);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.v16_full[i], 4);
            mbar_init(&sm.v16_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_most[i], 4);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.o_free[i], 4);
        }
        for (int i = 0; i < kNK; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < kNV; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 4);
        }
        mbar_init(&sm.drain, 1);
        sm.k_issued = sm.v_issued = 0;
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 13) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    int32_t *const ab = &sm.abort_flag;
    const Shape shape(L);

    if (warp < 8) {
        // ---------------- softmax ----------------
        const int a = warp >> 2; // half
        const int r = 128 * a + (tid & 127);
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_addr = tmem + lanes + a * kColS, o_addr = tmem + lanes + kColO + a * 128;
        uint32_t nt = 0, ns = 0; // tiles and blocks of this half so far
        for (uint32_t n = 0;; ++n) {
            if (!warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab))
                break;
            const Job &j = sm.job[n % kJobs];
            const int nblk = j.nblk, blk0 = j.blk0;
            if (nblk < 0)
                break;
            if (a >= halves(j)) {
                warp_arrive(&sm.job_empty[n % kJobs], lane);
                continue;
            }
            auto pos_of = [&](int row) { return shape.position(j.ctx, shape.token(j.row + row)); };
            const bool real = r < j.rows;
            const int pos = real ? pos_of(r) : -1;
            const int pos_lo = pos_of(128 * a), pos_hi = pos_of(min(j.rows, 128 * a + 128) - 1);
            if (!warp_wait(&sm.q_full[a], nt & 1u, ab))
                break;
            const float c = sm.c[a][nt & 1u][r & 127];
            const F2 cc = pack2(c, c);
            float m = kNoMax;
            F2 l[2] = {0ull, 0ull};
            bool ok = true;
            for (int k = 0; k < nblk; ++k, ++ns) {
                ok = warp_wait(&sm.s_full[a], ns & 1u, ab);
                if (!ok)
                    break;
                tc_fence_after();
                const int b0 = (blk0 + k) * kBlock;
                // Where some row does not see the whole block, the scores are masked in place first, which
                // keeps the masks out of every other block.
                if (b0 + kBlock - 1 > pos_lo || (L.window > 0 && b0 <= pos_hi - L.window)) {
                    const int w = L.window > 0 ? L.window : 0x7FFFFFFF;
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        const int d = pos - b0 - 32 * ch; // distance of the chunk's first key behind the token
                        uint32_t x[32];
                        tmem_ld32(s_addr + 32 * ch, x);
                        tmem_ld_wait(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (d < e || d - e >= w)
                                x[e] = 0xFF800000u;
                        tmem_st32(s_addr + 32 * ch, x);
                    }
                    tmem_st_wait();
                }
                uint32_t s[2][32]; // a chunk's scores arrive during the weights of the one before
                tmem_ld32(s_addr, s[0]);
                tmem_ld_wait(s[0]);
                float y = max32(s[0]) * c;
                bool any = __any_sync(kFull, y > m + kRaise);
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t (&x)[32] = s[ch & 1], (&next)[32] = s[(ch + 1) & 1];
                    if (any) {
                        const float mn = y > m + kRaise ? ceilf(y) : m, alpha = attn::ex2(m - mn);
                        m = mn;
                        l[0] = mul2(l[0], pack2(alpha, alpha));
                        l[1] = mul2(l[1], pack2(alpha, alpha));
                        rescale(o_addr, k > 0 ? 8 : 0, s_addr, ch, alpha);
                    }
                    if (ch < 3) // behind the call, which must not find a load on its way into registers
                        tmem_ld32(s_addr + 32 * (ch + 1), next);
                    const F2 nm = pack2(-m, -m);
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        if (e == 4 && ch == 3) {
                            tmem_st_wait();
                            tc_fence_before();
                            warp_arrive(&sm.p_most[a], lane);
                        }
                        if (e == 16 && ch < 3) { // the next chunk's maximum is found among these exponentials
                            tmem_ld_wait(next);
                            y = max32(next) * c;
                            any = __any_sync(kFull, y > m + kRaise);
                        }
                        float p0, p1;
                        unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), cc, nm), p0, p1);
                        p0 = attn::ex2(p0);
                        p1 = attn::ex2(p1);
                        l[(e >> 1) & 1] = add2(l[(e >> 1) & 1], pack2(p0, p1));
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p[e / 2]) : "f"(p1), "f"(p0));
                    }
                    tmem_st16(s_addr + 16 * ch, p); // over scores that have been read
                }
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&sm.p_full[a], lane);
            }
            if (!ok || !warp_wait(&sm.o_full[a], nt & 1u, ab))
                break;
            tc_fence_after();
            // ---- the end of the tile ----
            float *const part = j.slot >= 0 ? partial<kRows>(L, cta, j.slot) : nullptr;
            const int flat = j.row + r, tok = shape.token(flat);
            const int64_t at = (static_cast<int64_t>(j.tok0) + tok) * L.Hq + j.h * L.G + flat - tok * L.G;
            float l0, l1;
            unpack2(add2(l[0], l[1]), l0, l1);
            float *const mark = &sm.bad[a][nt % 3u][r & 127];
            const float sum = (l0 + l1) + *mark, inv = L.v_scale / sum;
            *mark = 0.f;
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t o[32];
                tmem_ld32(o_addr + 32 * ch, o);
                tmem_ld_wait(o);
                if (real && part != nullptr) {
                    float *dst = part + r * kHeadDim + 32 * ch;
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        store32(dst + e, o + e);
                } else if (real) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        w[e] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                    uint16_t *dst = L.O + at * kHeadDim + 32 * ch;
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        reinterpret_cast<uint4 *>(dst)[e / 4] = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                }
            }
            tc_fence_before();
            warp_arrive(&sm.o_free[a], lane);
            if (real && part != nullptr) {
                part[kRows * kHeadDim + r] = m;
                part[kRows * (kHeadDim + 1) + r] = sum;
            } else if (real && L.lse != nullptr) {
                L.lse[at] = (m + log2f(sum)) * 0.6931471805599453f;
            }
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            ++nt;
        }
    } else if (warp < 12) {
        // ---------------- queries; V to f16 ----------------
        const int t = tid - 256;
        uint32_t nt[2] = {0, 0}, c = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            ok = warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab);
            if (!ok)
                break;
            const Job j = sm.job[n % kJobs];
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            if (j.nblk < 0)
                break;
            for (int a = 0; ok && a < halves(j); ++a) {
                ok = warp_wait(&sm.q_empty[a], (nt[a] & 1u) ^ 1u, ab);
                if (!ok)
                    break;
                // a thread a row
                const int r = 128 * a + t, flat = j.row + r, tok = shape.token(flat);
                const bool real = r < j.rows;
                const uint4 *src = reinterpret_cast<const uint4 *>(L.Q + (static_cast<int64_t>(j.tok0) + tok) * L.q_st +
                                                                   static_cast<int64_t>(j.h * L.G + flat - tok * L.G) * L.q_sh);
                uint4 v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = real ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
                uint32_t e = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    e = __vmaxu2(__vmaxu2(__vmaxu2(e, v[i].x & 0x7F807F80u), __vmaxu2(v[i].y & 0x7F807F80u, v[i].z & 0x7F807F80u)), v[i].w & 0x7F807F80u);
                e = max(e >> 23, (e >> 7) & 0xFFu);
                const int sh = q_exp(e);
                const float up = exp2i(sh);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint2 a1, a2, b1, b2;
                    split_q8<Rest::kE5M2>(v[2 * i], up, a1, a2);
                    split_q8<Rest::kE5M2>(v[2 * i + 1], up, b1, b2);
                    const uint32_t at = attn::swz(t, i);
                    *reinterpret_cast<uint4 *>(sm.q[a][0] + at) = make_uint4(a1.x, a1.y, b1.x, b1.y);
                    *reinterpret_cast<uint4 *>(sm.q[a][1] + at) = make_uint4(a2.x, a2.y, b2.x, b2.y);
                }
                sm.c[a][nt[a] & 1u][t] = q_factor(e, L.score_scale);
                fence_proxy_async_smem();
                warp_arrive(&sm.q_full[a], lane);
                ++nt[a];
            }
            const int pos_lo = shape.position(j.ctx, shape.token(j.row));
            for (int k = 0; ok && k < j.nblk; ++k, ++c) {
                const uint32_t sv = c % kNV, slot = c & 1u;
                ok = warp_wait(&sm.v_full[sv], (c / kNV) & 1u, ab) && warp_wait(&sm.v16_empty[slot], ((c >> 1) & 1u) ^ 1u, ab);
                if (!ok)
                    break;
                // Values of keys that no row of the tile sees may be any bytes, NaN codes among them,
                // and zero times NaN is not zero: they enter as zeros.
                const int b0 = (j.blk0 + k) * kBlock;
                const bool edge = b0 < j.lo || b0 + kBlock > j.hi;
                // Nor where one token of the tile sees a key and another does not: there NaN leaves the
                // values and enters the sums of the rows that see it.
                if (b0 + kBlock - 1 > pos_lo || (L.window > 0 && b0 <= j.hi - 1 - L.window))
                    take_nan(sm.v[sv], t, b0, j.lo, j.hi, shape, j.ctx, j.row, j.rows, sm.bad[0][(nt[0] + 2u) % 3u], sm.bad[1][(nt[1] + 2u) % 3u]);
#pragma unroll 2
                for (int i = 0; i < 8; ++i) {
                    const int q = t + 128 * i, key = q >> 3, c16 = q & 7;
                    uint4 x = *reinterpret_cast<const uint4 *>(sm.v[sv] + key * 128 + c16 * 16);
                    if (edge && (b0 + key < j.lo || b0 + key >= j.hi))
                        x = make_uint4(0u, 0u, 0u, 0u);
                    uint4 h0, h1;
                    e4m3x16_to_f16(x, h0, h1);
                    uint8_t *const dst = sm.v16[slot][c16 >> 2];
                    const int j0 = (2 * c16) & 7;
                    // half of the threads store in the other order, so that eight of them meet all banks
                    const bool flip = c16 >= 4;
                    *reinterpret_cast<uint4 *>(dst + attn::swz(key, j0 + flip)) = flip ? h1 : h0;
                    *reinterpret_cast<uint4 *>(dst + attn::swz(key, j0 + 1 - flip)) = flip ? h0 : h1;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.v16_full[slot]);
                    mbar_arrive(&sm.v_empty[sv]);
                }
            }
        }
    } else {
        if (warp == 12) {
            // ---------------- load ----------------
            Pieces<kRows> pieces;
            pieces.begin(L, shape, cta, lane);
            auto fetch = [&](const Job &j, int k) { // slots of the 32 pages of job j from block k on, one a lane
                const int pg = 2 * (j.blk0 + k) + lane; // between the pages that hold a key of the tile
                return pg >= (j.lo >> 6) && pg <= ((j.hi - 1) >> 6) && pg < 2 * (j.blk0 + j.nblk) ? phys_slot(L, j.b, pg) : -1;
            };
            uint32_t c = 0;
            Job j;
            bool more = pieces.next(L, shape, cta, lane, j), ok = true;
            int ids = more ? fetch(j, 0) : -1;
            for (uint32_t n = 0; ok; ++n) {
                ok = warp_wait(&sm.job_empty[n % kJobs], ((n / kJobs) & 1u) ^ 1u, ab);
                if (!ok)
                    break;
                if (!more)
                    j.nblk = -1;
                if (lane == 0) {
                    sm.job[n % kJobs] = j;
                    mbar_arrive(&sm.job_full[n % kJobs]);
                }
                if (!more)
                    break;
                Job jn;
                int ids_n = -1, nxt = j.nblk > 16 ? fetch(j, 16) : -1;
                // the next job is formed, and its first page ids asked for, while copies are in flight
                const int ahead = min(j.nblk, kNV) - 1;
                for (int k = 0; k < j.nblk; ++k, ++c) {
                    if (k > 0 && (k & 15) == 0) {
                        ids = nxt;
                        if (k + 16 < j.nblk)
                            nxt = fetch(j, k + 16);
                    }
                    const int s0 = __shfl_sync(kFull, ids, 2 * (k & 15)), s1 = __shfl_sync(kFull, ids, 2 * (k & 15) + 1);
                    const uint32_t bytes = ((s0 >= 0) + (s1 >= 0)) * attn::kPageBytes;
                    const int y0 = (s0 * L.Hkv + j.h) * kPageTokens, y1 = (s1 * L.Hkv + j.h) * kPageTokens;
                    const uint32_t sk = c % kNK, sv = c % kNV;
                    ok = warp_wait(&sm.k_empty[sk], ((c / kNK) & 1u) ^ 1u, ab);
                    if (!ok)
                        break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sm.k_full[sk], bytes);
                        if (s0 >= 0)
                            tma_load_2d(sm.k[sk], &map_k, 0, y0, &sm.k_full[sk]);
                        if (s1 >= 0)
                            tma_load_2d(sm.k[sk] + attn::kPageBytes, &map_k, 0, y1, &sm.k_full[sk]);
                        sm.k_issued = c + 1;
                    }
                    __syncwarp();
                    ok = warp_wait(&sm.v_empty[sv], ((c / kNV) & 1u) ^ 1u, ab);
                    if (!ok)
                        break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sm.v_full[sv], bytes);
                        if (s0 >= 0)
                            bulk_g2s(sm.v[sv], L.V + static_cast<int64_t>(y0) * kHeadDim, attn::kPageBytes, &sm.v_full[sv]);
                        if (s1 >= 0)
                            bulk_g2s(sm.v[sv] + attn::kPageBytes, L.V + static_cast<int64_t>(y1) * kHeadDim, attn::kPageBytes, &sm.v_full[sv]);
                        sm.v_issued = c + 1;
                    }
                    __syncwarp();
                    if (k == ahead) {
                        more = pieces.next(L, shape, cta, lane, jn);
                        if (more)
                            ids_n = fetch(jn, 0);
                    }
                }
                j = jn;
                ids = ids_n;
            }
        } else if (warp == 13) {
            // ---------------- products ----------------
            // Of each half in turn: the products of the block before, begun when three quarters of its weights
            // are there (the wake-up and six of eight steps pass during the rest), then S of this one.  The P of a
            // block lies over the S it came from; the tensor core takes its work in order, so S of the
            // next block may follow the products that read P without a wait.
            const uint64_t dk = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024), dq = sdesc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
            const uint64_t dv = sdesc_sw128(smem_u32(sm.v16[0][0]), kBlock * 128, 1024);
            uint32_t c = 0, ns[2] = {0, 0}, nt[2] = {0, 0}; // blocks; products and tiles of each half
            bool ok = true;
            int pend = 0;                        // halves of block c - 1 whose products are still to come
            bool p_first = false, p_last = false; // that block is the first, the last of its tile
            auto products = [&](int a) {
                const uint32_t slot = (c - 1) & 1u;
                if (!warp_wait(&sm.v16_full[slot], ((c - 1) >> 1) & 1u, ab) ||
                    (p_first && !warp_wait(&sm.o_free[a], (nt[a] & 1u) ^ 1u, ab)) || !warp_wait(&sm.p_most[a], ns[a] & 1u, ab))
                    return false;
                tc_fence_after();
                const uint32_t o = tmem + kColO + a * 128, p = tmem + a * kColS;
                const uint64_t v = dv + ((slot * 2 * kBlock * 128) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 6; ++kk)
                        mma_f16_ts(o, p + 8 * kk, v + 128 * kk, kIdescO, kk > 0 || !p_first);
                }
                __syncwarp();
                if (!warp_wait(&sm.p_full[a], ns[a] & 1u, ab))
                    return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 6; kk < 8; ++kk)
                        mma_f16_ts(o, p + 8 * kk, v + 128 * kk, kIdescO, 1);
                    if (p_last)
                        mma_commit(&sm.o_full[a]);
                    if (a == pend - 1)
                        mma_commit(&sm.v16_empty[slot]);
                }
                __syncwarp();
                ++ns[a];
                nt[a] += p_last;
                return true;
            };
            uint32_t nq[2] = {0, 0};
            for (uint32_t n = 0; ok; ++n) {
                ok = warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab);
                if (!ok)
                    break;
                const Job &job = sm.job[n % kJobs];
                const int nblk = job.nblk, hv = halves(job);
                warp_arrive(&sm.job_empty[n % kJobs], lane);
                // the last products of the tile before
                for (int a = 0; ok && a < pend; ++a)
                    ok = products(a);
                pend = 0;
                if (nblk < 0)
                    break;
                for (int k = 0; ok && k < nblk; ++k) {
                    const uint32_t sk = c % kNK;
                    ok = warp_wait(&sm.k_full[sk], (c / kNK) & 1u, ab);
                    for (int a = 0; ok && a < hv; ++a) {
                        if (k > 0)
                            ok = products(a);
                        else
                            ok = warp_wait(&sm.q_full[a], nq[a]++ & 1u, ab);
                        if (!ok)
                            break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) // four steps of each query part
                                mma_f8_ss(tmem + a * kColS, dq + ((a * 2 * kHalf * 128 + (kk >> 2) * kHalf * 128 + (kk & 3) * 32) >> 4),
                                          dk + ((sk * kBlock * 128 + (kk & 3) * 32) >> 4), kk < 4 ? kIdescS : kIdescRest, kk > 0);
                            mma_commit(&sm.s_full[a]);
                            if (k == nblk - 1)
                                mma_commit(&sm.q_empty[a]);
                            if (a == hv - 1)
                                mma_commit(&sm.k_empty[sk]);
                        }
                        __syncwarp();
                    }
                    ++c;
                    pend = hv;
                    p_first = k == 0;
                    p_last = k == nblk - 1;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (sm.abort_flag != 0) {
        // Copies and products in flight land before the CTA leaves (bounded waits).
        if (tid == 0) {
            set_status(L.status, PW_ERR_TIMEOUT);
            const uint32_t nk = sm.k_issued, nv = sm.v_issued;
            for (uint32_t s = 0; s < kNK && s < nk; ++s)
                (void)mbar_wait(&sm.k_full[s], ((nk - 1 - s) / kNK) & 1u);
            for (uint32_t s = 0; s < kNV && s < nv; ++s)
                (void)mbar_wait(&sm.v_full[s], ((nv - 1 - s) / kNV) & 1u);
        }
        if (warp == 13) {
            if (elect_one()) {
                mma_commit(&sm.drain);
                (void)mbar_wait(&sm.drain, 0);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

} // namespace

size_t tiles_workspace() { return workspace_bytes<kRows>(); }

cudaError_t tiles_launch(ChunkLaunch &L, int sms, cudaStream_t st)
{
    const int ctas = ctas_for<kRows>(L, sms);
    CUtensorMap k;
    cudaError_t e = page_tensor(L.K, L, &k);
    const int smem = static_cast<int>(sizeof(TileSmem) + 1024);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_chunk_tiles, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    k_chunk_tiles<<<ctas, kThreads, smem, st>>>(L, k);
    e = cudaGetLastError();
    return e == cudaSuccess ? merge_launch<kRows>(L, ctas, st) : e;
}

} // namespace chunk
} // namespace pw
