// pw_chunk_decode.cu -- pw_chunk_attn for few rows: single tokens and drafted ones.
//
// Reading the cache is what takes the time, so keys are the long side of the products and nothing
// is unpacked: a block of 128 keys is the M = 128 operand of
//   S^T = K [q1 q2]        (M = keys, N = 2 NT, K = 128 dims; E4M3)
//   O^T += V^T [P1 P2 P3]  (M = dims, N = 3 NT, K = 128 keys; E4M3, V read as stored, MN-major)
// straight from the bytes that TMA landed.  Queries enter as two exact E4M3 parts (pw_chunk.cuh),
// weights as three, each the remainder of the one before times 2^4 and rounded to 4 significant
// bits: together 12 bits (a relative 2^-12, half the error of one f16) of a weight of at least 2^-6
// and an absolute 2^-18 below, at no more passes over V, since the parts lie side by side along N.
//
// The running maximum of a row is a reference that only has to keep its weights in range: it moves
// when a score exceeds it by more than 2^8 (256 stays inside E4M3's 448), to 2^4 below that score,
// so that the largest weight lies in [2^4, 2^8] and the absolute error of the small ones is 2^-22
// of it.  That costs one vote per block instead of a reduction over the keys, which lie along the
// threads here.
//
// Two groups of four softmax warps take blocks in turn (block c goes to group c % 2), each with its
// own S, P, accumulator, reference and sums; they meet at the end of a tile.
//
//   warp 0       load: page ids, TMA copies into the ring of K and V stages, job records
//   warp 1       the products
//   warps 2-3    the next tile's queries
//   warps 4-11   softmax (two groups), and the end of a tile
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pw_chunk.cuh"

namespace pw {
namespace chunk {
namespace {

constexpr int kThreads = 384;
constexpr int kJobs = 4;
constexpr int kMinBlocks = 1;
constexpr uint32_t kBarBoth = 3; // named barrier of the two softmax groups (theirs: 1 and 2)
constexpr float kRaise = 8.f; // a row's reference moves when a score exceeds it by more (base 2),
constexpr float kBelow = 4.f; // to this much below that score

template <int NT> constexpr int kStagesFor = NT == 16 ? 6 : 5;

template <int NT>
struct __align__(1024) DecSmem {
    static constexpr int kStages = kStagesFor<NT>;
    uint8_t k[kStages][kBlock * 128]; // 128 keys x 128 dims
    uint8_t v[kStages][kBlock * 128];
    uint8_t p[2][3 * NT * 128];       // [group][part, row][key]
    uint8_t q[2][2 * NT * 128];       // [tile % 2][part, row][dim]
    float stage[NT][128];             // group 1's accumulator at the end of a tile
    float2 cm[2][NT];                 // [group]: score factor and reference of a row
    float red[2][4][NT];              // [group][warp]: block maxima, row sums
    float c[2][NT];                   // [tile % 2]: score factor
    int pos[2][NT];                   // [tile % 2]: position of the row's token
    Job job[kJobs];
    Plan plan;
    uint64_t job_full[kJobs], job_empty[kJobs];
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kStages], v_full[kStages], st_empty[kStages];
    uint64_t s_done[2], s_free[2], p_ready[2], pv_done[2];
    uint64_t drain;
    uint32_t issued; // blocks whose copies were issued
    uint32_t tmem;
    int32_t abort_flag;
};

// One key's weights of two rows: three E4M3 parts each (byte 0: the first row's), the second and
// third scaled by 2^4 and 2^8.
__device__ __forceinline__ void split3(float p0, float p1, uint32_t &a, uint32_t &b, uint32_t &c)
{
    float y0, y1;
    a = e4m3x2(p0, p1);
    e4m3x2_to_f32(a, y0, y1);
    p0 = (p0 - y0) * 16.f;
    p1 = (p1 - y1) * 16.f;
    b = e4m3x2(p0, p1);
    e4m3x2_to_f32(b, y0, y1);
    c = e4m3x2((p0 - y0) * 16.f, (p1 - y1) * 16.f);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Waits for this thread's tcgen05.ld; the registers pass through it, so that no use moves before.
__device__ __forceinline__ void tmem_wait8(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_decode(const ChunkLaunch L, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using Smem = DecSmem<NT>;
    constexpr int kSt = Smem::kStages;
    constexpr uint32_t kTmemCols = NT == 16 ? 256 : 512;
    constexpr uint32_t kColO = 4 * NT; // S of the two groups, then their accumulators
    constexpr uint32_t kIdescS = idesc_e4m3_f32(128, 2 * NT);
    constexpr uint32_t kIdescO = idesc_e4m3_f32(128, 3 * NT) | (1u << 15); // A (V^T) MN-major
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&sm.job_full[i], 1);
            mbar_init(&sm.job_empty[i], 2 + 1 + 8); // query, product and softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 2);
            mbar_init(&sm.q_empty[i], 1 + 8); // products, softmax warps
            mbar_init(&sm.s_done[i], 1);
            mbar_init(&sm.s_free[i], 4);
            mbar_init(&sm.p_ready[i], 4);
            mbar_init(&sm.pv_done[i], 1);
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
    if (warp == 1) {
        tmem_alloc(&sm.tmem, kTmemCols);
        tmem_relinquish();
    }
    make_plan<NT>(L, sm.plan, cta, kMinBlocks);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    int32_t *const ab = &sm.abort_flag;

    if (warp == 0) {
        // ---------------- load ----------------
        Pieces<NT> pieces;
        pieces.begin(L, sm.plan, reinterpret_cast<Cut *>(L.workspace), cta, lane);
        uint32_t c = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            Job j;
            const bool more = pieces.next(L, j);
            if (!more)
                j.nblk = -1;
            ok = warp_wait(&sm.job_empty[n % kJobs], ((n / kJobs) & 1u) ^ 1u, ab);
            if (!ok)
                break;
            if (lane == 0) {
                sm.job[n % kJobs] = j;
                mbar_arrive(&sm.job_full[n % kJobs]);
            }
            if (!more)
                break;
            const int plo = j.lo >> 6, phi = (j.hi - 1) >> 6; // pages that hold a key of the tile
            const int p0 = 2 * j.blk0;
            auto fetch = [&](int k) { // slots of the 32 pages from block k on, one a lane
                const int pg = p0 + 2 * k + lane;
                return pg >= plo && pg <= phi && pg < p0 + 2 * j.nblk ? phys_slot(L, j.b, pg) : -1;
            };
            int ids = fetch(0), nxt = fetch(16);
            for (int k = 0; k < j.nblk; ++k, ++c) {
                if (k > 0 && (k & 15) == 0) {
                    ids = nxt;
                    nxt = fetch(k + 16);
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
            }
        }
    } else if (warp == 1) {
        // ---------------- products ----------------
        // S of block c goes out before the products of block c - 2, the last block of the same
        // group: its S is read by then, so it computes while that group forms its weights.
        const uint64_t dk = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024), dv = sdesc_sw128(smem_u32(sm.v[0]), 16, 1024);
        const uint64_t dq = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024), dp = sdesc_sw128(smem_u32(sm.p[0]), 16, 1024);
        uint32_t c = 0;
        bool ok = true;
        // products of block cc, the first of its group in the tile or not
        auto pv = [&](uint32_t cc, bool first) {
            const uint32_t g = cc & 1u, s = cc % kSt;
            if (!warp_wait(&sm.v_full[s], (cc / kSt) & 1u, ab) || !warp_wait(&sm.p_ready[g], (cc >> 1) & 1u, ab))
                return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f8_ss(tmem + kColO + g * 3 * NT, dv + ((s * kBlock * 128 + kk * 32 * 128) >> 4),
                              dp + ((g * 3 * NT * 128 + kk * 32) >> 4), kIdescO, kk > 0 || !first);
                mma_commit(&sm.pv_done[g]);
                mma_commit(&sm.st_empty[s]);
            }
            __syncwarp();
            return true;
        };
        for (uint32_t n = 0; ok; ++n) {
            ok = warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab);
            if (!ok)
                break;
            const int nblk = sm.job[n % kJobs].nblk;
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            if (nblk < 0)
                break;
            const uint32_t qb = n & 1u;
            ok = warp_wait(&sm.q_full[qb], (n >> 1) & 1u, ab);
            for (int k = 0; ok && k < nblk + 2; ++k) {
                if (k < nblk) {
                    const uint32_t cc = c + k, g = cc & 1u, s = cc % kSt;
                    ok = warp_wait(&sm.k_full[s], (cc / kSt) & 1u, ab) && warp_wait(&sm.s_free[g], ((cc >> 1) & 1u) ^ 1u, ab);
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
                if (k >= 2)
                    ok = pv(c + k - 2, k < 4);
            }
            c += nblk;
        }
    } else if (warp < 4) {
        // ---------------- queries ----------------
        const int half = lane >> 4, l = lane & 15;
        for (uint32_t n = 0;; ++n) {
            if (!warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab))
                break;
            const Job j = sm.job[n % kJobs];
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            if (j.nblk < 0)
                break;
            const uint32_t qb = n & 1u;
            if (!warp_wait(&sm.q_empty[qb], ((n >> 1) & 1u) ^ 1u, ab))
                break;
            const Sequence s = sequence(L, j.b);
            for (int r = 2 * (warp - 2) + half; r < NT; r += 4) {
                const int flat = j.row + r, tok = flat / L.G;
                const bool real = r < j.rows;
                const uint16_t *row = real ? L.Q + (static_cast<int64_t>(j.tok0) + tok) * L.q_st +
                                                 static_cast<int64_t>(j.h * L.G + flat - tok * L.G) * L.q_sh
                                           : nullptr;
                const float c = stage_q_row(row, sm.q[qb], r, NT + r, l, L.score_scale);
                if (l == 0) {
                    sm.c[qb][r] = c;
                    sm.pos[qb][r] = real ? position(s, tok) : -1;
                }
            }
            fence_proxy_async_smem();
            warp_arrive(&sm.q_full[qb], lane);
        }
    } else {
        // ---------------- softmax ----------------
        // A wait that fails is voted on at the group's next barrier, so that its four warps leave
        // together; a group that leaves, at the end of its work too, takes one turn at the barrier of
        // both groups (kBarBoth), where the other one learns of it.
        const uint32_t g = (warp >> 2) - 1, bar = 1 + g;
        const int qd = warp & 3, key = 32 * qd + lane; // this thread's key of a block, and dim of O^T
        const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t s_addr = tmem + lanes + g * 2 * NT, o_addr = tmem + lanes + kColO + g * 3 * NT;
        uint8_t *const pcol = sm.p[g] + (key & 15);
        uint32_t c = 0; // blocks of the CTA before this tile
        bool ok = true, both = false;
        for (uint32_t n = 0;; ++n) {
            ok = warp_wait(&sm.job_full[n % kJobs], (n / kJobs) & 1u, ab);
            if (bar_or(bar, 128, !ok))
                break;
            const Job j = sm.job[n % kJobs];
            warp_arrive(&sm.job_empty[n % kJobs], lane);
            if (j.nblk < 0)
                break;
            const uint32_t qb = n & 1u;
            ok = warp_wait(&sm.q_full[qb], (n >> 1) & 1u, ab);
            if (key < NT)
                sm.cm[g][key] = make_float2(sm.c[qb][key], kNoMax);
            if (bar_or(bar, 128, !ok))
                break;
            const int R8 = (j.rows + 7) >> 3;                                     // groups of eight rows
            const int pos_lo = sm.pos[qb][0], pos_hi = sm.pos[qb][j.rows - 1]; // first and last token
            float l[NT];
#pragma unroll
            for (int r = 0; r < NT; ++r)
                l[r] = 0.f;
            uint32_t used = 0, u = 0;
            bool failed = false;
            for (int k = static_cast<int>((c ^ g) & 1u); k < j.nblk; k += 2, ++used) {
                const uint32_t cc = c + k, s = cc % kSt;
                u = cc >> 1;
                const int b0 = (j.blk0 + k) * kBlock, kp = b0 + key; // this thread's position
                // some row does not see the whole block
                const bool edge = b0 + kBlock - 1 > pos_lo || (L.window > 0 && b0 <= pos_hi - L.window);
                ok = warp_wait(&sm.s_done[g], u & 1u, ab);
                tc_fence_after();
                float y[NT]; // base-2 exponents
                float top = -INFINITY;
#pragma unroll
                for (int r8 = 0; r8 < NT / 8; ++r8)
                    if (r8 < R8) {
                        uint32_t a[8], b[8];
                        tmem_ld8(s_addr + 8 * r8, a);
                        tmem_ld8(s_addr + NT + 8 * r8, b);
                        tmem_wait8(a);
                        tmem_wait8(b);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int r = 8 * r8 + e;
                            const float2 cm = sm.cm[g][r];
                            y[r] = (__uint_as_float(a[e]) + __uint_as_float(b[e])) * cm.x;
                            if (edge) {
                                const int pr = sm.pos[qb][r];
                                if (kp > pr || (L.window > 0 && kp <= pr - L.window))
                                    y[r] = -INFINITY;
                            }
                            if (r < j.rows)
                                top = fmaxf(top, y[r] - cm.y);
                        }
                    }
                tc_fence_before();
                warp_arrive(&sm.s_free[g], lane);
                if (bar_or(bar, 128, !ok || top > kRaise)) {
                    // The block's maximum of every row; where it exceeds the reference by more than
                    // kRaise, the reference moves and what the row has so far is scaled.
#pragma unroll
                    for (int r = 0; r < NT; ++r)
                        if (r < j.rows) {
                            float m = y[r];
#pragma unroll
                            for (int d = 16; d > 0; d >>= 1)
                                m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
                            if (lane == 0)
                                sm.red[g][qd][r] = m;
                        }
                    if (ok && used > 0) // the products so far
                        ok = warp_wait(&sm.pv_done[g], (u - 1) & 1u, ab);
                    if (bar_or(bar, 128, !ok)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int r8 = 0; r8 < NT / 8; ++r8)
                        if (r8 < R8) {
                            float alpha[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int r = 8 * r8 + e;
                                const float m = sm.cm[g][r].y;
                                const float top_r = fmaxf(fmaxf(sm.red[g][0][r], sm.red[g][1][r]),
                                                          fmaxf(sm.red[g][2][r], sm.red[g][3][r]));
                                alpha[e] = r < j.rows && top_r - m > kRaise ? attn::ex2(m - (top_r - kBelow)) : 1.f;
                                l[r] *= alpha[e];
                            }
                            if (used > 0) {
#pragma unroll
                                for (int part = 0; part < 3; ++part) {
                                    uint32_t o[8];
                                    tmem_ld8(o_addr + part * NT + 8 * r8, o);
                                    tmem_wait8(o);
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha[e]);
                                    tmem_st8(o_addr + part * NT + 8 * r8, o);
                                }
                            }
                        }
                    tmem_st_wait();
                    tc_fence_before();
                    bar_sync(bar, 128); // every thread has read the old references
                    if (key < j.rows) {
                        const float top_r = fmaxf(fmaxf(sm.red[g][0][key], sm.red[g][1][key]),
                                                  fmaxf(sm.red[g][2][key], sm.red[g][3][key]));
                        if (top_r - sm.cm[g][key].y > kRaise)
                            sm.cm[g][key].y = top_r - kBelow;
                    }
                    bar_sync(bar, 128);
                }
                // the group's last products have read its weights (and, at a tile's start, the
                // previous tile's accumulator has been read)
                if (cc >= 2)
                    ok = warp_wait(&sm.pv_done[g], (u - 1) & 1u, ab);
                uint32_t off[8]; // this key's byte in rows 0..7 of a swizzle atom
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    off[e] = static_cast<uint32_t>(e * 128 + (((key >> 4) ^ e) << 4));
#pragma unroll
                for (int r8 = 0; r8 < NT / 8; ++r8)
                    if (r8 < R8) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const int r = 8 * r8 + e;
                            const float p0 = attn::ex2(y[r] - sm.cm[g][r].y), p1 = attn::ex2(y[r + 1] - sm.cm[g][r + 1].y);
                            l[r] += p0;
                            l[r + 1] += p1;
                            uint32_t w[3];
                            split3(p0, p1, w[0], w[1], w[2]);
#pragma unroll
                            for (int part = 0; part < 3; ++part) {
                                uint8_t *const at = pcol + (part * NT + 8 * r8) * 128;
                                at[off[e]] = static_cast<uint8_t>(w[part]);
                                at[off[e + 1]] = static_cast<uint8_t>(w[part] >> 8);
                            }
                        }
                    }
                // Values of keys that no row of the tile sees may be any bytes, NaN codes among them,
                // and zero times NaN is not zero: they become zeros before the products read them.
                if (b0 < j.lo || b0 + kBlock > j.hi) {
                    ok = warp_wait(&sm.v_full[s], (cc / kSt) & 1u, ab) && ok;
                    if (kp < j.lo || kp >= j.hi) {
                        uint4 *row = reinterpret_cast<uint4 *>(sm.v[s] + key * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            row[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&sm.p_ready[g], lane);
            }
            if (failed)
                break;
            // ---- the end of the tile: sums over the keys, group 1's part to group 0, the result ----
            if (ok && used > 0)
                ok = warp_wait(&sm.pv_done[g], u & 1u, ab);
            tc_fence_after();
            float o[NT];
#pragma unroll
            for (int r8 = 0; r8 < NT / 8; ++r8) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[8 * r8 + e] = 0.f;
                if (r8 < R8 && used > 0) {
                    uint32_t a[8], b[8], d[8];
                    tmem_ld8(o_addr + 8 * r8, a);
                    tmem_ld8(o_addr + NT + 8 * r8, b);
                    tmem_ld8(o_addr + 2 * NT + 8 * r8, d);
                    tmem_wait8(a);
                    tmem_wait8(b);
                    tmem_wait8(d);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[8 * r8 + e] = fmaf(fmaf(__uint_as_float(d[e]), 0.0625f, __uint_as_float(b[e])), 0.0625f,
                                             __uint_as_float(a[e]));
                }
            }
            tc_fence_before();
#pragma unroll
            for (int r = 0; r < NT; ++r)
                if (r < j.rows) {
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1)
                        l[r] += __shfl_xor_sync(kFull, l[r], d);
                    if (lane == 0)
                        sm.red[g][qd][r] = l[r];
                    if (g == 1)
                        sm.stage[r][key] = o[r];
                }
            if (bar_or(kBarBoth, 256, !ok)) {
                both = true;
                break;
            }
            float *part = j.slot >= 0 ? partial<NT>(L, cta, j.slot) : nullptr;
            if (g == 0) {
#pragma unroll
                for (int r = 0; r < NT; ++r)
                    if (r < j.rows) {
                        const float m0 = sm.cm[0][r].y, m1 = sm.cm[1][r].y, m = fmaxf(m0, m1);
                        const float a0 = attn::ex2(m0 - m), a1 = attn::ex2(m1 - m);
                        const float sum = a0 * ((sm.red[0][0][r] + sm.red[0][1][r]) + (sm.red[0][2][r] + sm.red[0][3][r])) +
                                          a1 * ((sm.red[1][0][r] + sm.red[1][1][r]) + (sm.red[1][2][r] + sm.red[1][3][r]));
                        const float v = a0 * o[r] + a1 * sm.stage[r][key];
                        if (part != nullptr) {
                            part[r * kHeadDim + key] = v;
                            if (key == r) {
                                part[NT * kHeadDim + r] = m;
                                part[NT * (kHeadDim + 1) + r] = sum;
                            }
                        } else {
                            const int flat = j.row + r, tok = flat / L.G;
                            const int64_t at = (static_cast<int64_t>(j.tok0) + tok) * L.Hq + j.h * L.G + flat - tok * L.G;
                            L.O[at * kHeadDim + key] = __bfloat16_as_ushort(__float2bfloat16_rn(v * (L.v_scale / sum)));
                            if (L.lse != nullptr && key == r)
                                L.lse[at] = (m + log2f(sum)) * 0.6931471805599453f;
                        }
                    }
            }
            warp_arrive(&sm.q_empty[qb], lane); // positions and factors read
            bar_sync(kBarBoth, 256); // group 0 has read the staged part and the references
            c += j.nblk;
        }
        if (!both)
            (void)bar_or(kBarBoth, 256, true);
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
        if (warp == 1) {
            if (elect_one()) {
                mma_commit(&sm.drain);
                (void)mbar_wait(&sm.drain, 0);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int NT>
cudaError_t launch(const ChunkLaunch &L, int ctas, cudaStream_t st)
{
    static_assert(sizeof(DecSmem<NT>) + 1024 <= 227 * 1024, "shared-memory layout too large");
    CUtensorMap k, v;
    cudaError_t e = page_tensor(L.K, L, &k);
    if (e == cudaSuccess)
        e = page_tensor(L.V, L, &v);
    const int smem = static_cast<int>(sizeof(DecSmem<NT>) + 1024);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_chunk_decode<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    k_chunk_decode<NT><<<ctas, kThreads, smem, st>>>(L, k, v);
    e = cudaGetLastError();
    return e == cudaSuccess ? merge_launch<NT>(L, ctas, st) : e;
}

} // namespace

size_t decode_workspace(int rows) { return rows <= 16 ? workspace_bytes<16>() : workspace_bytes<32>(); }

cudaError_t decode_launch(const ChunkLaunch &L, int rows, int ctas, cudaStream_t st)
{
    return rows <= 16 ? launch<16>(L, ctas, st) : launch<32>(L, ctas, st);
}

} // namespace chunk
} // namespace pw
