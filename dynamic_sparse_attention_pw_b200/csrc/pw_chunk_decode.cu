// pw_chunk_decode.cu -- pw_chunk_attn for few rows: single tokens and drafted ones.
//
// Reading the cache is what takes the time, so keys are the long side of the products and nothing
// is unpacked: a block of 128 keys is the M = 128 operand of
//   S^T = K [q1 q2]        (M = keys, N = 2 NT, K = 128 dims; E4M3)
//   O^T += V^T [P1 P2 P3]  (M = dims, N = 3 NT, K = 128 keys; E4M3, V read as stored, MN-major)
// straight from the bytes that TMA landed.  Queries enter as two E4M3 parts, q2 times 2^5 (pw_chunk.cuh),
// weights, rounded to f16, as three exact ones: four significant bits, the next four of what is left,
// and the rest, at no more passes over V, since the parts lie side by side along N.  A weight of at
// most 1 whose f16 bits are shifted right by 7 is the E4M3 code of 2^8 times the weight, cut off, with
// the subnormal numbers of both formats in the same places, so a part is a shift and a subtraction.
// Four rows' codes of a key go out in one store: exponentials, parts and stores of a block took 461
// cycles with conversions and a store a code, 260 so.
//
// The running maximum of a row is a reference that only has to keep its weights in range: it lies
// above the scores and moves when one exceeds it, to 2 (base 2) above that score, so that a row's
// largest weight lies in [2^-2, 1] and a weight below f16's normal range (2^-14) is off by at most half of
// its smallest step, 2^-25, or 2^-23 of the largest.  That costs one vote per block instead of a reduction over
// the keys, which lie along the threads here.  Moves further up are fewer, and lose more: 4 above, a
// row of 128k keys that together make 3% beside one key could lose all of them (decode 64 ragged / 4 x 128k /
// verify 32 x 5: 4 above 205 / 179 / 95 us, 2 above 206 / 180 / 98, 1 above 208 / 181 / 101).
//
// Two CTAs share an SM, each with its own stretch of the work, so that one computes while the other
// starts or ends a tile.  The two softmax warps that share a quarter of the keys share the rows: four of
// every eight each, and the halves never wait for each other.  Code that a tile runs once (its first
// block, its end) is kept short: at the start of a call it runs from a cold instruction cache, and
// unrolled over the rows it alone took 14 us.
//
//   warps 0-7    softmax, and the end of a tile
//   warp 8       load: page ids, TMA copies into the ring of K and V stages, job records
//   warp 9       the products
//   warp 10      the next tile's queries
//
// What bounds it: the bytes of the cache.  64 sequences of 500 to 16k tokens, 8 query heads a kv head
// (1.1 GB): 196 to 207 us (B200s differ), 5.4 to 5.6 TB/s with launch and merge; four of 128k: 174 to
// 182 us, 5.9 to 6.2 TB/s (a copy: 6.55).  With 20 rows (5 drafted tokens, 4 heads) the weights'
// arithmetic takes longer than the bytes: 32 sequences of 1k to 8k 96 to 98 us, 3.1 TB/s (tiles of 32 rows
// for them: 105 us).  Small calls are latency: 16.4 us for one token over 2k keys.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pw_chunk.cuh"

namespace pw {
namespace chunk {
namespace {

constexpr int kThreads = 352;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpQ = 10;
constexpr int kJobs = 4;
// Query tiles: S runs up to one block, so up to one tile, ahead of the products, and a tile's slot is
// free when its results are written.
constexpr int kQ = 2;
constexpr float kAbove = 2.f;  // a row's reference moves to this much above its largest score (base 2)

template <int NT> constexpr int kStagesFor = NT == 16 ? 3 : 2;
template <int NT> constexpr int kCols = (3 * NT + 15) / 16 * 16; // columns of the weights: a whole number of cores

template <int NT>
struct __align__(1024) DecSmem {
    static constexpr int kStages = kStagesFor<NT>;
    uint8_t k[kStages][kBlock * 128]; // 128 keys x 128 dims
    uint8_t v[kStages][kBlock * 128];
    // the weights as a matrix of 3 NT columns (part, row; a few of padding behind) by 128 keys, columns
    // contiguous: cores of 8 keys by 16 columns (128 bytes), the cores of the same 8 keys side by side
    uint8_t p[kCols<NT> * 128];
    uint8_t q[kQ][2 * NT * 128];      // [tile % kQ][part, row][dim]
    float c[kQ][NT];                  // [tile % kQ]: factor of a row's scores
    int pos[kQ][NT];                  // [tile % kQ]: position of the row's token
    int at[kQ][NT];                   // [tile % kQ]: its row of O and lse
    float nm[NT];                     // a row's reference, negated
    float alpha[NT];                  // factor when it moves
    float red[4][NT];                 // [key quarter]: block maxima, row sums
    float bad[kQ][NT];                // [tile % kQ]: NaN for a row that sees a value taken out as NaN, else 0
    Job job[kJobs];
    uint64_t job_full[kJobs], job_empty[kJobs];
    uint64_t q_full[kQ], q_empty[kQ];
    uint64_t k_full[kStages], v_full[kStages], st_empty[kStages];
    uint64_t s_done[2], s_free[2], p_ready, pv_done;
    uint64_t drain;
    uint32_t issued; // blocks whose copies were issued
    uint32_t tmem;
    int32_t abort_flag;
};

// One key's weights of two rows, 0..1, rounded to f16 and cut exactly into three E4M3 parts each, the
// second and third times 2^4 and 2^8: bits 7..14 and 23..30 of w hold the codes of the two rows.
__device__ __forceinline__ void split3(float p0, float p1, uint32_t (&w)[3])
{
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(p1), "f"(p0));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t cut = w[i] & 0xFF80FF80u;
        const __half2 rest = __hsub2(*reinterpret_cast<const __half2 *>(&w[i]), *reinterpret_cast<const __half2 *>(&cut));
        const __half2 r = __hmul2(rest, __float2half2_rn(16.f));
        w[i + 1] = *reinterpret_cast<const uint32_t *>(&r);
    }
}

__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// One key's values without their NaN; the rows that see the key (position kp) get one.  Rare, and so not
// inlined.
static __device__ __noinline__ void take_nan(uint4 *row, int kp, const int *pos, float *bad, int rows, int window)
{
    bool has = false;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        uint4 x = row[i];
        if (drop_nan(x)) {
            row[i] = x;
            has = true;
        }
    }
    if (has)
#pragma unroll 1
        for (int r = 0; r < rows; ++r)
            if (pos[r] >= kp && (window == 0 || pos[r] - kp < window))
                bad[r] = __int_as_float(0x7FC00000);
}

// Waits for this thread's tcgen05.ld; the registers pass through it, so that no use moves before.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[4])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])::"memory");
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 2)
    k_chunk_decode(const ChunkLaunch L, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using Smem = DecSmem<NT>;
    constexpr int kSt = Smem::kStages;
    constexpr uint32_t kTmemCols = NT == 16 ? 128 : 256;
    constexpr uint32_t kColO = 4 * NT; // two S, then the accumulator
    constexpr uint32_t kIdescS = idesc_e4m3_f32(128, 2 * NT);
    constexpr uint32_t kIdescO = idesc_e4m3_f32(128, kCols<NT>) | (1u << 15) | (1u << 16); // A (V^T) and B (P) MN-major
    constexpr int kKeys8 = kCols<NT> * 8; // bytes of P of 8 keys
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;

    allow_merge();
    if (tid == 0) {
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&sm.job_full[i], 1);
            mbar_init(&sm.job_empty[i], 1 + 1 + 8); // query, product and softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_done[i], 1);
            mbar_init(&sm.s_free[i], 8);
        }
        mbar_init(&sm.p_ready, 8);
        mbar_init(&sm.pv_done, 1);
        for (int i = 0; i < kQ; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1 + 8); // products, softmax warps
        }
        for (int i = 0; i < kSt; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.st_empty[i], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.issued = 0;
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&sm.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    int32_t *const ab = &sm.abort_flag;
    const Shape shape(L);

    if (warp < kWarpLoad) {
        // ---------------- softmax ----------------
        // A wait that fails is voted on at the next barrier of the half, so that its four warps leave
        // together; the other half finds the abort flag.
        const uint32_t h4 = 4 * (warp >> 2), bar = 1 + (warp >> 2);
        const int qd = warp & 3, key = 32 * qd + lane; // this thread's key of a block, and dim of O^T
        // its rows: 8 i + h4 + e, for e in 0..3 and i in 0..R8 - 1
        const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t o_addr = tmem + lanes + kColO + h4;
        uint8_t *const pcol = sm.p + (key >> 3) * kKeys8 + (key & 7) * 16;
        const float *const nm = sm.nm + h4, *const alpha = sm.alpha + h4;
        uint32_t c = 0; // blocks of the CTA before this tile
        bool ok = true;
        for (uint32_t n = 0;; ++n) {
            ok = warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab);
            if (bar_or(bar, 128, !ok))
                break;
            const Job &job = sm.job[n % kJobs];
            const int nblk = job.nblk, blk0 = job.blk0, lo = job.lo, hi = job.hi, rows = job.rows, slot = job.slot;
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            if (nblk < 0)
                break;
            const uint32_t qb = n % kQ;
            ok = warp_wait(&sm.q_full[qb], (n / kQ) & 1u, ab);
            if (key < NT && ((key ^ h4) & 4) == 0)
                sm.nm[key] = key < rows ? -kNoMax : 0.f; // rows of padding score 0 and never move
            if (bar_or(bar, 128, !ok))
                break;
            const int R8 = max(rows - static_cast<int>(h4) + 7, 0) >> 3;    // this half's groups of four rows
            const int pos_lo = sm.pos[qb][0], pos_hi = sm.pos[qb][rows - 1]; // first and last token
            const float *const fac = sm.c[qb] + h4;
            F2 l[NT / 8][2];
#pragma unroll
            for (int i = 0; i < NT / 8; ++i)
                l[i][0] = l[i][1] = 0ull;
            bool failed = false;
            for (int k = 0; k < nblk; ++k) {
                const uint32_t cc = c + k, s = cc % kSt, g = cc & 1u, s_addr = tmem + lanes + g * 2 * NT + h4;
                const int b0 = (blk0 + k) * kBlock, kp = b0 + key; // this thread's position
                ok = warp_wait(&sm.s_done[g], (cc >> 1) & 1u, ab);
                tc_fence_after();
                F2 y[NT / 8][2]; // base-2 exponents
                bool over = false;
#pragma unroll
                for (int i0 = 0; i0 < NT / 8; i0 += 2)
                    if (i0 < R8) {
                        uint32_t a[2][4], b[2][4];
#pragma unroll
                        for (int i = 0; i < 2 && i0 + i < NT / 8; ++i) {
                            tmem_ld4(s_addr + 8 * (i0 + i), a[i]);
                            tmem_ld4(s_addr + NT + 8 * (i0 + i), b[i]);
                        }
#pragma unroll
                        for (int i = 0; i < 2 && i0 + i < NT / 8; ++i) {
                            tmem_wait(a[i]);
                            tmem_wait(b[i]);
                        }
#pragma unroll
                        for (int i = 0; i < 2 && i0 + i < NT / 8; ++i) {
                            const float4 f = *reinterpret_cast<const float4 *>(fac + 8 * (i0 + i));
                            const F2 down = pack2(1.f / kRestUp, 1.f / kRestUp);
                            y[i0 + i][0] = mul2(fma2(pack2(__uint_as_float(b[i][0]), __uint_as_float(b[i][1])), down,
                                                     pack2(__uint_as_float(a[i][0]), __uint_as_float(a[i][1]))), pack2(f.x, f.y));
                            y[i0 + i][1] = mul2(fma2(pack2(__uint_as_float(b[i][2]), __uint_as_float(b[i][3])), down,
                                                     pack2(__uint_as_float(a[i][2]), __uint_as_float(a[i][3]))), pack2(f.z, f.w));
                        }
                    }
                tc_fence_before();
                warp_arrive(&sm.s_free[g], lane);
                // some row does not see the whole block
                const bool edge = b0 + kBlock - 1 > pos_lo || (L.window > 0 && b0 <= pos_hi - L.window);
                if (edge) {
#pragma unroll
                    for (int i = 0; i < NT / 8; ++i)
                        if (i < R8) {
                            const int4 pr = *reinterpret_cast<const int4 *>(sm.pos[qb] + 8 * i + h4);
                            const int w = L.window > 0 ? L.window : 0x7FFFFFFF; // key kp is seen from kp to kp + w - 1
                            float x0, x1;
                            unpack2(y[i][0], x0, x1);
                            x0 = pr.x >= kp && pr.x - kp < w ? x0 : -INFINITY;
                            x1 = pr.y >= kp && pr.y - kp < w ? x1 : -INFINITY;
                            y[i][0] = pack2(x0, x1);
                            unpack2(y[i][1], x0, x1);
                            x0 = pr.z >= kp && pr.z - kp < w ? x0 : -INFINITY;
                            x1 = pr.w >= kp && pr.w - kp < w ? x1 : -INFINITY;
                            y[i][1] = pack2(x0, x1);
                        }
                }
#pragma unroll
                for (int i = 0; i < NT / 8; ++i)
                    if (i < R8) {
                        const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(nm + 8 * i);
                        float x0, x1, x2, x3;
                        unpack2(add2(y[i][0], m.x), x0, x1);
                        unpack2(add2(y[i][1], m.y), x2, x3);
                        over = over || fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) > 0.f;
                    }
                if (bar_or(bar, 128, !ok || over)) {
                    // The block's maximum of every row; where it exceeds the reference, the reference
                    // moves and what the row has so far is scaled.
#pragma unroll
                    for (int i = 0; i < NT / 8; ++i)
                        if (i < R8) {
                            float4 m;
                            unpack2(y[i][0], m.x, m.y);
                            unpack2(y[i][1], m.z, m.w);
                            m = make_float4(warp_max(m.x), warp_max(m.y), warp_max(m.z), warp_max(m.w));
                            if (lane == 0)
                                *reinterpret_cast<float4 *>(&sm.red[qd][8 * i + h4]) = m;
                        }
                    if (ok && k > 0) // the products so far
                        ok = warp_wait(&sm.pv_done, (cc - 1) & 1u, ab);
                    if (bar_or(bar, 128, !ok)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    if (key < NT && ((key ^ h4) & 4) == 0) { // a thread a row
                        const float top = fmaxf(fmaxf(sm.red[0][key], sm.red[1][key]), fmaxf(sm.red[2][key], sm.red[3][key]));
                        const float m = sm.nm[key];
                        const bool move = key < rows && top + m > 0.f;
                        sm.alpha[key] = move ? attn::ex2(-(top + kAbove) - m) : 1.f;
                        if (move)
                            sm.nm[key] = -(top + kAbove);
                    }
                    bar_sync(bar, 128);
#pragma unroll
                    for (int i = 0; i < NT / 8; ++i)
                        if (i < R8) {
                            const ulonglong2 al = *reinterpret_cast<const ulonglong2 *>(alpha + 8 * i);
                            l[i][0] = mul2(l[i][0], al.x);
                            l[i][1] = mul2(l[i][1], al.y);
                        }
                    if (k > 0) {
#pragma unroll 1
                        for (int i = 0; i < R8; ++i) {
                            const float4 al = *reinterpret_cast<const float4 *>(alpha + 8 * i);
                            if (al.x * al.y * al.z * al.w == 1.f) // none of the four moves (a factor is 1 or at most 2^-kAbove)
                                continue;
#pragma unroll 1
                            for (int part = 0; part < 3; ++part) {
                                const uint32_t at = o_addr + part * NT + 8 * i;
                                uint32_t o[4];
                                tmem_ld4(at, o);
                                tmem_wait(o);
                                o[0] = __float_as_uint(__uint_as_float(o[0]) * al.x);
                                o[1] = __float_as_uint(__uint_as_float(o[1]) * al.y);
                                o[2] = __float_as_uint(__uint_as_float(o[2]) * al.z);
                                o[3] = __float_as_uint(__uint_as_float(o[3]) * al.w);
                                tmem_st4(at, o);
                            }
                        }
                        tmem_st_wait();
                        tc_fence_before();
                    }
                }
                // the last products have read their weights
                if (cc >= 1)
                    ok = warp_wait(&sm.pv_done, (cc - 1) & 1u, ab);
#pragma unroll
                for (int i = 0; i < NT / 8; ++i)
                    if (i < R8) {
                        const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(nm + 8 * i);
                        uint32_t w[2][3];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float p0, p1;
                            unpack2(add2(y[i][e], e == 0 ? m.x : m.y), p0, p1);
                            p0 = attn::ex2(p0);
                            p1 = attn::ex2(p1);
                            l[i][e] = add2(l[i][e], pack2(p0, p1));
                            split3(p0, p1, w[e]);
                        }
#pragma unroll
                        for (int part = 0; part < 3; ++part) { // the codes of the four rows
                            const int n = part * NT + 8 * i;   // first column of the eight
                            *reinterpret_cast<uint32_t *>(pcol + n / 16 * 128 + n % 16 + h4) =
                                attn::prmt(w[0][part] >> 7, w[1][part] >> 7, 0x6420u);
                        }
                    }
                // Values of keys that no row of the tile sees may be any bytes, NaN codes among them,
                // and zero times NaN is not zero: they become zeros before the products read them.
                if (h4 == 0 && (b0 < lo || b0 + kBlock > hi)) {
                    ok = warp_wait(&sm.v_full[s], (cc / kSt) & 1u, ab) && ok;
                    if (kp < lo || kp >= hi) {
                        uint4 *row = reinterpret_cast<uint4 *>(sm.v[s] + key * 128);
#pragma unroll 1
                        for (int i = 0; i < 8; ++i)
                            row[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                // Nor where one token of the tile sees a key and another does not: there NaN leaves the
                // values and enters the sums of the rows that see it.
                if (h4 == 0 && edge && pos_lo != pos_hi) {
                    ok = warp_wait(&sm.v_full[s], (cc / kSt) & 1u, ab) && ok;
                    take_nan(reinterpret_cast<uint4 *>(sm.v[s] + key * 128), kp, sm.pos[qb], sm.bad[qb], rows, L.window);
                }
                fence_proxy_async_smem();
                warp_arrive(&sm.p_ready, lane);
            }
            if (failed)
                break;
            // ---- the end of the tile ----
            // Sums over the 32 keys of a warp: a lane gives half of its rows away twice, then the
            // lanes that hold the same row add up.
#pragma unroll
            for (int i = 0; i < NT / 8; ++i)
                if (i < R8) {
                    float x0, x1, x2, x3;
                    unpack2(l[i][0], x0, x1);
                    unpack2(l[i][1], x2, x3);
                    const bool up = lane & 16, odd = lane & 8;
                    const float k0 = up ? x2 : x0, k1 = up ? x3 : x1;
                    const float y0 = k0 + __shfl_xor_sync(kFull, up ? x0 : x2, 16), y1 = k1 + __shfl_xor_sync(kFull, up ? x1 : x3, 16);
                    float z = (odd ? y1 : y0) + __shfl_xor_sync(kFull, odd ? y0 : y1, 8);
                    z += __shfl_xor_sync(kFull, z, 4);
                    z += __shfl_xor_sync(kFull, z, 2);
                    z += __shfl_xor_sync(kFull, z, 1);
                    if ((lane & 7) == 0)
                        sm.red[qd][8 * i + h4 + (lane >> 3)] = z;
                }
            if (ok)
                ok = warp_wait(&sm.pv_done, (c + nblk - 1) & 1u, ab);
            if (bar_or(bar, 128, !ok))
                break;
            tc_fence_after();
            float *const part = slot >= 0 ? partial<NT>(L, cta, slot) : nullptr;
#pragma unroll 1
            for (int i = 0; i < R8; ++i) {
                const int r = 8 * i + h4; // rows r to r + 3
                uint32_t x[4], y[4], z[4];
                tmem_ld4(o_addr + 8 * i, x);
                tmem_ld4(o_addr + NT + 8 * i, y);
                tmem_ld4(o_addr + 2 * NT + 8 * i, z);
                tmem_wait(x);
                tmem_wait(y);
                tmem_wait(z);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r + e < rows) {
                        const int rr = r + e;
                        const float v = fmaf(fmaf(__uint_as_float(z[e]), 0x1p-4f, __uint_as_float(y[e])), 0x1p-4f, __uint_as_float(x[e])) * 0x1p-8f;
                        const float sum = ((sm.red[0][rr] + sm.red[1][rr]) + (sm.red[2][rr] + sm.red[3][rr])) + sm.bad[qb][rr];
                        if (part != nullptr) {
                            part[rr * kHeadDim + key] = v;
                            if (key == 0) {
                                part[NT * kHeadDim + rr] = -sm.nm[rr];
                                part[NT * (kHeadDim + 1) + rr] = sum;
                            }
                        } else {
                            const int64_t at = sm.at[qb][rr];
                            L.O[at * kHeadDim + key] = __bfloat16_as_ushort(__float2bfloat16_rn(v * (L.v_scale / sum)));
                            if (L.lse != nullptr && key == 0)
                                L.lse[at] = (log2f(sum) - sm.nm[rr]) * 0.6931471805599453f;
                        }
                    }
            }
            tc_fence_before();
            warp_arrive(&sm.q_empty[qb], lane); // positions, places and factors read
            bar_sync(bar, 128);                 // references and sums read
            c += nblk;
        }
    } else if (warp == kWarpLoad) {
        // ---------------- load ----------------
        Pieces<NT> pieces;
        pieces.begin(L, shape, cta, lane);
        // slots of the 32 pages of job j from block k on, one a lane
        auto fetch = [&](const Job &j, int k) {
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
            const int ahead = min(j.nblk, kSt) - 1;
            for (int k = 0; k < j.nblk; ++k, ++c) {
                if (k > 0 && (k & 15) == 0) {
                    ids = nxt;
                    if (k + 16 < j.nblk)
                        nxt = fetch(j, k + 16);
                }
                const int s0 = __shfl_sync(kFull, ids, 2 * (k & 15)), s1 = __shfl_sync(kFull, ids, 2 * (k & 15) + 1);
                const uint32_t s = c % kSt;
                ok = warp_wait(&sm.st_empty[s], ((c / kSt) & 1u) ^ 1u, ab);
                if (!ok)
                    break;
                if (lane == 0) {
                    const uint32_t bytes = ((s0 >= 0) + (s1 >= 0)) * attn::kPageBytes;
                    const int y0 = (s0 * L.Hkv + j.h) * kPageTokens, y1 = (s1 * L.Hkv + j.h) * kPageTokens;
                    mbar_arrive_expect_tx(&sm.k_full[s], bytes);
                    if (s0 >= 0)
                        tma_load_2d(sm.k[s], &map_k, 0, y0, &sm.k_full[s]);
                    if (s1 >= 0)
                        tma_load_2d(sm.k[s] + attn::kPageBytes, &map_k, 0, y1, &sm.k_full[s]);
                    mbar_arrive_expect_tx(&sm.v_full[s], bytes);
                    if (s0 >= 0)
                        tma_load_2d(sm.v[s], &map_v, 0, y0, &sm.v_full[s]);
                    if (s1 >= 0)
                        tma_load_2d(sm.v[s] + attn::kPageBytes, &map_v, 0, y1, &sm.v_full[s]);
                    sm.issued = c + 1;
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
    } else if (warp == kWarpMma) {
        // ---------------- products ----------------
        // S of block c goes out before the products of block c - 1, also across the end of a tile, so
        // that it is there when the softmax comes to it.
        const uint64_t dk = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024), dv = sdesc_sw128(smem_u32(sm.v[0]), 16, 1024);
        const uint64_t dq = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024), dp = sdesc_plain(smem_u32(sm.p), kKeys8, 128);
        uint32_t c = 0;
        bool ok = true;
        // products of block cc, the first of its tile or not
        auto pv = [&](uint32_t cc, bool first) {
            const uint32_t s = cc % kSt;
            if (!warp_wait(&sm.v_full[s], (cc / kSt) & 1u, ab) || !warp_wait(&sm.p_ready, cc & 1u, ab))
                return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f8_ss(tmem + kColO, dv + ((s * kBlock * 128 + kk * 32 * 128) >> 4), dp + ((kk * 4 * kKeys8) >> 4), kIdescO,
                              kk > 0 || !first);
                mma_commit(&sm.pv_done);
                mma_commit(&sm.st_empty[s]);
            }
            __syncwarp();
            return true;
        };
        bool f1 = false; // block c - 1 is the first of its tile
        for (uint32_t n = 0; ok; ++n) {
            ok = warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab);
            if (!ok)
                break;
            const int nblk = sm.job[n % kJobs].nblk;
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            const uint32_t qb = n % kQ;
            if (nblk >= 0)
                ok = warp_wait(&sm.q_full[qb], (n / kQ) & 1u, ab);
            // behind the last job: the products that are left
            for (int k = 0; ok && k < (nblk >= 0 ? nblk : 1); ++k, ++c) {
                if (nblk >= 0) {
                    const uint32_t g = c & 1u, s = c % kSt;
                    ok = warp_wait(&sm.k_full[s], (c / kSt) & 1u, ab) && warp_wait(&sm.s_free[g], ((c >> 1) & 1u) ^ 1u, ab);
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f8_ss(tmem + g * 2 * NT, dk + ((s * kBlock * 128 + kk * 32) >> 4),
                                      dq + ((qb * 2 * NT * 128 + kk * 32) >> 4), kIdescS, kk > 0);
                        mma_commit(&sm.s_done[g]);
                        if (k == nblk - 1)
                            mma_commit(&sm.q_empty[qb]);
                    }
                    __syncwarp();
                }
                if (c >= 1)
                    ok = pv(c - 1, f1);
                f1 = k == 0;
            }
            if (nblk < 0)
                break;
        }
    } else if (warp == kWarpQ) {
        // ---------------- queries ----------------
        const int half = lane >> 4, l = lane & 15;
        for (uint32_t n = 0;; ++n) {
            if (!warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab))
                break;
            const Job j = sm.job[n % kJobs];
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            if (j.nblk < 0)
                break;
            const uint32_t qb = n % kQ;
            if (!warp_wait(&sm.q_empty[qb], ((n / kQ) & 1u) ^ 1u, ab))
                break;
            // sixteen lanes a row, four rows of a half-warp at a time
#pragma unroll 1
            for (int r0 = half; r0 < NT; r0 += 8) {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = r0 + 2 * i, flat = j.row + r, tok = shape.token(flat), head = j.h * L.G + flat - tok * L.G;
                    const bool real = r < j.rows;
                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (real)
                        v[i] = __ldg(reinterpret_cast<const uint4 *>(L.Q + (static_cast<int64_t>(j.tok0) + tok) * L.q_st +
                                                                     static_cast<int64_t>(head) * L.q_sh) + l);
                    if (l == 0) {
                        sm.pos[qb][r] = real ? shape.position(j.ctx, tok) : -1;
                        sm.at[qb][r] = (j.tok0 + tok) * L.Hq + head;
                        sm.bad[qb][r] = 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = r0 + 2 * i;
                    const float c = stage_q_row(v[i], sm.q[qb], r, NT + r, l, L.score_scale);
                    if (l == 0)
                        sm.c[qb][r] = c;
                }
            }
            fence_proxy_async_smem();
            warp_arrive(&sm.q_full[qb], lane);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (sm.abort_flag != 0) {
        // Copies and products in flight land before the CTA leaves (bounded waits).
        if (tid == 0) {
            set_status(L.status, PW_ERR_TIMEOUT);
            const uint32_t n = sm.issued;
            for (uint32_t s = 0; s < kSt && s < n; ++s) {
                const uint32_t last = s + (n - 1 - s) / kSt * kSt;
                (void)mbar_wait(&sm.k_full[s], (last / kSt) & 1u);
                (void)mbar_wait(&sm.v_full[s], (last / kSt) & 1u);
            }
        }
        if (warp == kWarpMma) {
            if (elect_one()) {
                mma_commit(&sm.drain);
                (void)mbar_wait(&sm.drain, 0);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int NT>
cudaError_t launch(ChunkLaunch &L, int sms, cudaStream_t st)
{
    const int ctas = ctas_for<NT>(L, sms);
    static_assert(sizeof(DecSmem<NT>) + 1024 <= 113 * 1024, "shared-memory layout too large");
    CUtensorMap k, v;
    cudaError_t e = page_tensor(L.K, L, &k);
    if (e == cudaSuccess)
        e = page_tensor(L.V, L, &v);
    const int smem = static_cast<int>(sizeof(DecSmem<NT>) + 1024);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_chunk_decode<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) // room for both CTAs of an SM
        e = cudaFuncSetAttribute(k_chunk_decode<NT>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess)
        return e;
    k_chunk_decode<NT><<<ctas, kThreads, smem, st>>>(L, k, v);
    e = cudaGetLastError();
    return e == cudaSuccess ? merge_launch<NT>(L, ctas, st) : e;
}

} // namespace

size_t decode_workspace(int rows) { return rows <= 16 ? workspace_bytes<16>() : rows <= 24 ? workspace_bytes<24>() : workspace_bytes<32>(); }

cudaError_t decode_launch(ChunkLaunch &L, int rows, int sms, cudaStream_t st)
{
    return rows <= 16 ? launch<16>(L, sms, st) : rows <= 24 ? launch<24>(L, sms, st) : launch<32>(L, sms, st);
}

} // namespace chunk
} // namespace pw
