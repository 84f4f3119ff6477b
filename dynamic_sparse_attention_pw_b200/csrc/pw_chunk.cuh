// pw_chunk.cuh -- what the two kernels of pw_chunk_attn share: how the work is cut into tiles and
// dealt out to the CTAs, the partial results of tiles that several CTAs work on, bounded waits.
//
// Work.  The rows of a sequence and kv head are its tokens times the G query heads that share the
// kv head, flat index token * G + head.  A tile is NT consecutive rows; its keys (the union of what
// its rows see) are cut into blocks of 128 positions, two pages.  All blocks of all tiles form one
// line, ordered by (sequence, kv head, tile, block), and the CTAs take equal stretches of it, so
// one long context, many short ones and any mixture fill the GPU alike.  The lengths are read
// on the device, by the load warp of every CTA for itself.
//
// A tile that lies within one stretch is finished by its CTA.  One that is cut leaves partial
// results (fp32 accumulator, running maximum, sum) in the workspace, at most two of a CTA: the end
// of a tile that an earlier CTA began (slot 0) and the beginning of one that goes on (slot 1).
// k_chunk_merge joins them in CTA order, so the result does not depend on timing.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pw_attn_common.cuh"
#include "pw_tokens.cuh"

namespace pw {
namespace chunk {

using namespace tokens;

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kSms = 148;
// CTAs of a kernel: small tiles two an SM, large ones one.
template <int NT>
__host__ __device__ constexpr int max_ctas() { return NT <= 32 ? 2 * kSms : kSms; }
constexpr int kBlock = 128;    // keys per block
constexpr float kNoMax = -1e30f; // running maximum of a row that has seen no key

// What the tiles of a call depend on besides their sequence.
struct Shape {
    int G, window, last; // last position a page table's row can hold
    uint32_t mul, shift; // n / G = (n * mul / 2^32 + n) >> shift

    __device__ __forceinline__ explicit Shape(const ChunkLaunch &L)
        : G(L.G), window(L.window), last(L.pm.max_pages * kPageTokens - 1), mul(L.g_mul), shift(L.g_shift)
    {
    }
    __device__ __forceinline__ int token(int row) const // of a flat row
    {
        const uint32_t n = static_cast<uint32_t>(row);
        return static_cast<int>((__umulhi(n, mul) + n) >> shift);
    }
    __device__ __forceinline__ int position(int ctx, int token) const
    {
        return static_cast<int>(min(static_cast<uint32_t>(ctx) + static_cast<uint32_t>(token), static_cast<uint32_t>(last)));
    }
};

struct Sequence {
    int row0; // first row of Q (token) of the sequence
    int qlen; // new tokens
    int ctx;  // tokens before them
};

// Contents that the arguments rule out (offsets outside [0, T] or falling, a negative context, a
// position outside the table's row) are recorded and clamped, so that nothing is addressed outside
// the caller's buffers.
__device__ __forceinline__ Sequence sequence(const ChunkLaunch &L, int b)
{
    const int T = static_cast<int>(L.tb.T);
    const int c0 = __ldg(L.tb.cu + b), c1 = __ldg(L.tb.cu + b + 1);
    const int ctx = L.tb.ctx != nullptr ? __ldg(L.tb.ctx + b) : 0;
    Sequence s;
    s.row0 = min(max(c0, 0), T);
    s.qlen = max(min(max(c1, 0), T) - s.row0, 0);
    s.ctx = max(ctx, 0);
    const int64_t end = static_cast<int64_t>(s.ctx) + s.qlen, room = static_cast<int64_t>(L.pm.max_pages) * kPageTokens;
    if (c0 != s.row0 || c1 != s.row0 + s.qlen || (s.qlen > 0 && (ctx < 0 || end > room)))
        set_status(L.status, PW_ERR_INVALID_ARG);
    return s;
}

struct Tile {
    int row, rows;  // flat rows of the sequence and kv head
    int lo, hi;     // keys [lo, hi) that some row of it sees
    int blk0, nblk; // their blocks
};

template <int NT>
__device__ __forceinline__ Tile tile_of(const Shape &p, int qlen, int ctx, int i)
{
    Tile t;
    t.row = i * NT;
    t.rows = min(qlen * p.G - t.row, NT);
    t.hi = p.position(ctx, p.token(t.row + t.rows - 1)) + 1;
    t.lo = p.window > 0 ? max(p.position(ctx, p.token(t.row)) - p.window + 1, 0) : 0;
    t.blk0 = t.lo / kBlock;
    t.nblk = (t.hi + kBlock - 1) / kBlock - t.blk0;
    return t;
}

template <int NT>
__device__ __forceinline__ int tiles_of(const Shape &p, int qlen)
{
    return (qlen * p.G + NT - 1) / NT;
}

// Blocks of one kv head of each lane's sequence.  A lane counts a few tiles by itself, the warp those
// of a sequence of many together.  Not inlined: it runs once or twice, from a cold instruction cache.
template <int NT>
__device__ __noinline__ int64_t head_blocks(const Shape p, int qlen, int ctx, int lane)
{
    constexpr int kAlone = 2;
    const int tiles = tiles_of<NT>(p, qlen);
    int64_t n = 0;
    for (uint32_t many = __ballot_sync(kFull, tiles > kAlone), first = 1; first != 0u || many != 0u; first = 0) {
        // the first round: every lane its own few tiles; the others: a sequence of many
        const int from = first != 0u ? lane : __ffs(many) - 1;
        const int q = __shfl_sync(kFull, qlen, from), c = __shfl_sync(kFull, ctx, from), e = __shfl_sync(kFull, tiles, from);
        const bool alone = first != 0u;
        int64_t m = 0;
        for (int i = alone ? 0 : lane, end = alone && e > kAlone ? 0 : e; i < end; i += alone ? 1 : 32)
            m += tile_of<NT>(p, q, c, i).nblk;
        if (alone) {
            n = m;
            continue;
        }
        many &= many - 1;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            m += __shfl_xor_sync(kFull, m, d);
        if (lane == from)
            n = m;
    }
    return n;
}

// The line of all blocks in equal stretches, the first `longer` of them one block longer.
struct Stretches {
    int64_t len;
    int longer, ctas;

    __device__ __forceinline__ int64_t begin(int j) const { return len * j + min(j, longer); }
};

// One piece of a tile, as the roles of a CTA hand it on.
struct Job {
    int nblk;      // blocks of the piece; -1: no more
    int blk0;      // first of them
    int lo, hi;    // the tile's keys
    int row, rows; // the tile's rows
    int b, h;
    int tok0;      // Q row of the sequence's first token
    int ctx;       // its position
    int slot;      // -1: the whole tile, 0 / 1: partial
};

// Where the tile that stretch j starts in was cut, for k_chunk_merge.
struct Cut {
    Stretches all;
    int64_t ts, te; // first block of the tile and the one behind its last
    int inside;     // the stretch starts behind the tile's first block
    int row, rows, h, tok0;
};

template <int NT>
__host__ __device__ constexpr size_t partial_floats() { return static_cast<size_t>(NT) * (kHeadDim + 2); }

constexpr size_t kCutBytes = (sizeof(Cut) * 2 * kSms + 255) / 256 * 256;

template <int NT>
__host__ __device__ constexpr size_t workspace_bytes() { return kCutBytes + 2 * max_ctas<NT>() * partial_floats<NT>() * sizeof(float); }

// Partial of CTA j, slot s: acc [NT][128], then max [NT], then sum [NT].
template <int NT>
__device__ __forceinline__ float *partial(const ChunkLaunch &L, int j, int s)
{
    return reinterpret_cast<float *>(static_cast<uint8_t *>(L.workspace) + kCutBytes) +
           (static_cast<size_t>(j) * 2 + s) * partial_floats<NT>();
}

// The pieces of a CTA's stretch, one after the other; a warp runs it (uniformly).
template <int NT>
struct Pieces {
    Stretches all;
    int64_t x, x1;
    int b, h, i, off; // next piece: tile i of (b, h), from its block off on
    Sequence s;
    int tiles;
    bool first;

    __device__ __forceinline__ void begin(const ChunkLaunch &L, const Shape &p, int cta, int lane)
    {
        const int B = L.tb.B, grid = gridDim.x;
        // All blocks, 32 sequences at a time; the first 32 counts stay.  (Four groups of loads at once hid
        // their latency in large batches, but the code of it cost a small call more.)
        int64_t mine = 0, total = 0;
#pragma unroll 1
        for (int base = 0; base < B; base += 32) {
            const Sequence q = base + lane < B ? sequence(L, base + lane) : Sequence{0, 0, 0};
            const int64_t n = head_blocks<NT>(p, q.qlen, q.ctx, lane);
            total += n;
            if (base == 0)
                mine = n;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            total += __shfl_xor_sync(kFull, total, d);
        total *= L.Hkv;
        all.ctas = static_cast<int>(min(static_cast<int64_t>(grid), max(total, static_cast<int64_t>(1))));
        all.len = grid == 1 ? total : total < grid ? min(total, static_cast<int64_t>(1)) : static_cast<int64_t>(__umul64hi(total, L.ctas_mul));
        all.longer = total < grid ? 0 : static_cast<int>(total - all.len * grid);
        x = cta < all.ctas ? all.begin(cta) : total;
        x1 = cta < all.ctas ? all.begin(cta + 1) : total;
        first = true;
        if (x >= x1) {
            none(L, cta, lane);
            return;
        }
        // the sequence and head that x lies in
        int64_t rest = x, per_head = 1;
        b = -1;
        for (int base = 0; b < 0 && base < B; base += 32) {
            int64_t n = mine;
            if (base > 0) {
                const Sequence q = base + lane < B ? sequence(L, base + lane) : Sequence{0, 0, 0};
                n = head_blocks<NT>(p, q.qlen, q.ctx, lane);
            }
            int64_t incl = n * L.Hkv;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(kFull, incl, d);
                if (lane >= d)
                    incl += o;
            }
            const uint32_t beyond = __ballot_sync(kFull, incl > rest);
            if (beyond != 0u) {
                const int k = __ffs(beyond) - 1;
                b = base + k;
                per_head = __shfl_sync(kFull, n, k);
                rest -= __shfl_sync(kFull, incl - n * L.Hkv, k);
            } else {
                rest -= __shfl_sync(kFull, incl, 31);
            }
        }
        if (b < 0) { // cannot happen while the lengths stay as they were
            none(L, cta, lane);
            return;
        }
        for (h = 0;; h += 32) { // heads that end at or before x
            const int k = __popc(__ballot_sync(kFull, (h + lane + 1) * per_head <= rest));
            if (k < 32) {
                h += k;
                break;
            }
        }
        rest -= h * per_head;
        s = sequence(L, b);
        tiles = tiles_of<NT>(p, s.qlen);
        for (i = 0;; i += 32) { // 32 tiles at a time
            const int n = i + lane < tiles ? tile_of<NT>(p, s.qlen, s.ctx, i + lane).nblk : 0;
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kFull, incl, d);
                if (lane >= d)
                    incl += o;
            }
            const uint32_t beyond = __ballot_sync(kFull, incl > rest);
            if (beyond != 0u) {
                const int k = __ffs(beyond) - 1;
                i += k;
                off = static_cast<int>(rest) - __shfl_sync(kFull, incl - n, k);
                return;
            }
            if (i + 32 >= tiles) { // as above
                none(L, cta, lane);
                return;
            }
            rest -= __shfl_sync(kFull, incl, 31);
        }
    }

    __device__ __forceinline__ void none(const ChunkLaunch &L, int cta, int lane)
    {
        x = x1;
        if (lane == 0)
            static_cast<Cut *>(L.workspace)[cta].inside = 0;
    }

    __device__ __forceinline__ bool next(const ChunkLaunch &L, const Shape &p, int cta, int lane, Job &j)
    {
        if (x >= x1)
            return false;
        const Tile t = tile_of<NT>(p, s.qlen, s.ctx, i);
        const int n = static_cast<int>(min(static_cast<int64_t>(t.nblk - off), x1 - x));
        j = Job{n, t.blk0 + off, t.lo, t.hi, t.row, t.rows, b, h, s.row0, s.ctx, off > 0 ? 0 : (n < t.nblk ? 1 : -1)};
        if (first && lane == 0)
            static_cast<Cut *>(L.workspace)[cta] = Cut{all, x - off, x - off + t.nblk, off > 0, t.row, t.rows, h, s.row0};
        first = false;
        x += n;
        off = 0;
        if (++i == tiles) {
            i = 0;
            if (++h == L.Hkv) {
                h = 0;
                while (x < x1 && ++b < L.tb.B) {
                    s = sequence(L, b);
                    tiles = tiles_of<NT>(p, s.qlen);
                    if (tiles > 0)
                        break;
                }
                if (b >= L.tb.B)
                    x = x1;
            }
        }
        return true;
    }
};

// ---------------------------------------------------------------------------------------
// Bounded waits: a CTA whose wait runs out raises its abort flag, which ends every other wait in it.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The whole warp waits and agrees, in step: lanes that spin apart cost 1 to 2% of the kernels' time, and
// one lane that waits for all a quarter and more.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int32_t *abort_flag)
{
    if (__all_sync(kFull, mbar_try_wait(bar, parity)))
        return true;
    const long long t0 = clock64();
    for (;;) {
        if (__all_sync(kFull, mbar_try_wait(bar, parity)))
            return true;
        bool over = *reinterpret_cast<volatile int32_t *>(abort_flag) != 0;
        if (clock64() - t0 > kWaitCycles) {
            *reinterpret_cast<volatile int32_t *>(abort_flag) = 1;
            over = true;
        }
        if (__any_sync(kFull, over))
            return false;
    }
}

__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane)
{
    __syncwarp();
    if (lane == 0)
        mbar_arrive(bar);
}

__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t n, bool pred)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 q, %1, 0;\n\t"
                 "bar.red.or.pred p, %2, %3, q;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(r)
                 : "r"(pred ? 1u : 0u), "r"(id), "r"(n)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t n)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// ---------------------------------------------------------------------------------------
// Queries: a row times the power of two that brings its largest magnitude into [128, 256), split
// into two 8-bit parts.  The first is the nearest E4M3 value.  Of the 8 significant bits of a bf16 value
// that leaves 3 (the rest is at most half a step), so that the second needs range rather than bits:
//   Rest::kE5M2     the rest as E5M2 (3 bits, steps down to 2^-16), where both parts are summed in
//                   one accumulator: their products differ in the instruction's operand type alone;
//   Rest::kE4M3Up5  2^5 times the rest as E4M3 (4 bits, steps down to 2^-9), where the parts have accumulators
//                   of their own and a factor costs nothing.
// Either sum is exact for every element within 2^13 of the row's largest (the first part keeps its four bits
// down to 2^-6); below, it is off by at most 2^-14 (2^-15), 2^-21 (2^-22) of the largest.  With the rest as plain
// E4M3, whose steps end at 2^-9, an element 2^13 below the largest was off by up to 2^-4 of itself.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t max_exp8(const uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max((w[i] >> 7) & 0xFFu, (w[i] >> 23) & 0xFFu));
    return m;
}

__device__ __forceinline__ int q_exp(uint32_t e) { return min(max(134 - static_cast<int>(e), -126), 126); }
__device__ __forceinline__ float exp2i(int s) { return __int_as_float((s + 127) << 23); }

__device__ __forceinline__ void e4m3x2_to_f32(uint32_t pair, float &lo, float &hi)
{
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(pair)));
    const __half2 h = *reinterpret_cast<const __half2 *>(&h2);
    lo = __low2float(h);
    hi = __high2float(h);
}

enum class Rest { kE5M2, kE4M3Up5 };
constexpr float kRestUp = 32.f; // kE4M3Up5

// Two f32 -> packed E5M2 pair (round to nearest even); `lo` lands in the low byte.
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

template <Rest kRest>
__device__ __forceinline__ void split_q8(const uint4 v, float scale, uint2 &q1, uint2 &q2)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x0 = bf16_lo(w[i]) * scale, x1 = bf16_hi(w[i]) * scale;
        a[i] = e4m3x2(x0, x1);
        float y0, y1;
        e4m3x2_to_f32(a[i], y0, y1);
        b[i] = kRest == Rest::kE5M2 ? e5m2x2(x0 - y0, x1 - y1) : e4m3x2((x0 - y0) * kRestUp, (x1 - y1) * kRestUp);
    }
    q1 = make_uint2(a[0] | (a[1] << 16), a[2] | (a[3] << 16));
    q2 = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
}

// The factor that takes the score of a row's parts to a base-2 exponent, from the row's largest
// exponent; NaN for a row that holds an infinity or NaN, so that its output is NaN.  Kept above zero, so
// that a masked score (-infinity) stays one in a row of zeros.
__device__ __forceinline__ float q_factor(uint32_t e, float score_scale)
{
    return e == 255u ? __int_as_float(0x7FC00000) : fmaxf(score_scale * exp2i(-q_exp(e)), 1e-30f);
}

// Sixteen lanes of a half-warp (l = lane % 16) bring one row: its two parts (kE4M3Up5) into rows r1 and r2 of a
// K-major operand tile (128-byte rows, 128-byte swizzle).  Returns the row's factor.
// v: the lane's eight elements.
__device__ __forceinline__ float stage_q_row(const uint4 v, uint8_t *tile, int r1, int r2, int l, float score_scale)
{
    uint32_t e = max_exp8(v);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1)
        e = max(e, __shfl_xor_sync(kFull, e, d));
    const int s = q_exp(e);
    uint2 q1, q2;
    split_q8<Rest::kE4M3Up5>(v, exp2i(s), q1, q2);
    const int in = (l & 1) * 8;
    *reinterpret_cast<uint2 *>(tile + attn::swz(r1, l >> 1) + in) = q1;
    *reinterpret_cast<uint2 *>(tile + attn::swz(r2, l >> 1) + in) = q2;
    return q_factor(e, score_scale);
}

// Bytes of w that hold the E4M3 code of NaN, as 0xFF each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u) * 0xFFu; }

// Takes the NaN codes out of a chunk of values; whether there were any.
__device__ __forceinline__ bool drop_nan(uint4 &x)
{
    const uint4 n = make_uint4(nan_bytes(x.x), nan_bytes(x.y), nan_bytes(x.z), nan_bytes(x.w));
    x = make_uint4(x.x & ~n.x, x.y & ~n.y, x.z & ~n.z, x.w & ~n.w);
    return (n.x | n.y | n.z | n.w) != 0u;
}

// Physical slot of a page, checked; 0 where the entry is bad (recorded).
__device__ __forceinline__ int phys_slot(const ChunkLaunch &L, int b, int page)
{
    const int p = page < L.pm.max_pages ? __ldg(L.pm.table + static_cast<int64_t>(b) * L.pm.max_pages + page) : -1;
    if (p < 0 || p >= L.pm.n_phys) {
        set_status(L.status, PW_ERR_INVALID_ARG);
        return 0;
    }
    return p;
}

// A cache as a 2-D byte tensor [n_phys * Hkv * 64][128] in boxes of one page with the 128-byte
// swizzle, so that one copy lands a page as a matrix operand.
cudaError_t page_tensor(const uint8_t *pages, const ChunkLaunch &L, CUtensorMap *map);

cudaError_t decode_launch(ChunkLaunch &L, int rows, int sms, cudaStream_t st);
size_t decode_workspace(int rows);
cudaError_t tiles_launch(ChunkLaunch &L, int sms, cudaStream_t st);
size_t tiles_workspace();

// Joins the partial results of the tiles that were cut: block j does the tile that stretch j starts
// inside of, unless an earlier stretch starts inside of it too.  A warp has NT / 64 rows (one of a
// small tile).  Behind the kernel for few rows, which leaves registers, the blocks are brought up while
// it still runs (programmatic launch) and wait for its end: 128 threads of 64 registers fit beside it.
template <int NT>
__global__ void __launch_bounds__(128, 8) k_chunk_merge(const ChunkLaunch L)
{
    constexpr int kR = NT <= 64 ? 1 : NT / 64;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int j = blockIdx.x, lane = threadIdx.x & 31, r0 = (blockIdx.y * 4 + (threadIdx.x >> 5)) * kR;
    // Records are read as they lie there and never trusted for an address: where two calls share a
    // workspace against the rules, the results are wrong, but nothing outside the buffers is touched.
    const Cut c = reinterpret_cast<const Cut *>(L.workspace)[j];
    const int ctas = min(c.all.ctas, static_cast<int>(gridDim.x)), rows = min(c.rows, NT);
    if (c.inside != 1 || j == 0 || r0 >= rows || c.all.begin(j - 1) > c.ts)
        return;
    int n = 1; // pieces: slot 1 of CTA j - 1, slot 0 of CTAs j .. j + n - 2
    while (j + n - 1 < ctas && c.all.begin(j + n - 1) < c.te)
        ++n;
    const float *first = partial<NT>(L, j - 1, 1), *rest = partial<NT>(L, j, 0);
    auto piece = [&](int i) { return i == 0 ? first : rest + static_cast<size_t>(i - 1) * 2 * partial_floats<NT>(); };
    float top[kR], sum[kR];
    float4 acc[kR];
#pragma unroll
    for (int e = 0; e < kR; ++e) {
        top[e] = -INFINITY;
        for (int i = lane; i < n; i += 32)
            top[e] = fmaxf(top[e], piece(i)[NT * kHeadDim + r0 + e]);
    }
#pragma unroll
    for (int e = 0; e < kR; ++e) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], d));
        sum[e] = 0.f;
        acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i0 = 0; i0 < n; i0 += 32) {
        float w[kR];
#pragma unroll
        for (int e = 0; e < kR; ++e) {
            w[e] = 0.f;
            if (i0 + lane < n) {
                const float *p = piece(i0 + lane);
                w[e] = attn::ex2(p[NT * kHeadDim + r0 + e] - top[e]);
                sum[e] += w[e] * p[NT * (kHeadDim + 1) + r0 + e];
            }
        }
        const int m = min(32, n - i0);
#pragma unroll(kR == 1 ? 8 : 2)
        for (int i = 0; i < m; ++i) {
            const float4 *o = reinterpret_cast<const float4 *>(piece(i0 + i) + r0 * kHeadDim) + lane;
#pragma unroll
            for (int e = 0; e < kR; ++e) {
                const float wi = __shfl_sync(kFull, w[e], i);
                const float4 v = o[e * (kHeadDim / 4)];
                acc[e].x = fmaf(wi, v.x, acc[e].x);
                acc[e].y = fmaf(wi, v.y, acc[e].y);
                acc[e].z = fmaf(wi, v.z, acc[e].z);
                acc[e].w = fmaf(wi, v.w, acc[e].w);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kR; ++e) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum[e] += __shfl_xor_sync(kFull, sum[e], d);
        if (r0 + e >= rows)
            break;
        const float inv = L.v_scale / sum[e];
        const int flat = c.row + r0 + e, tok = Shape(L).token(flat);
        const int64_t at = (static_cast<int64_t>(c.tok0) + tok) * L.Hq + static_cast<int64_t>(c.h) * L.G + flat - tok * L.G;
        if (at < 0 || at >= L.tb.T * L.Hq)
            break;
        const __nv_bfloat162 a = __floats2bfloat162_rn(acc[e].x * inv, acc[e].y * inv), b = __floats2bfloat162_rn(acc[e].z * inv, acc[e].w * inv);
        reinterpret_cast<uint2 *>(L.O + at * kHeadDim)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        if (L.lse != nullptr && lane == 0)
            L.lse[at] = (top[e] + log2f(sum[e])) * 0.6931471805599453f;
    }
}

// Lets k_chunk_merge come up; every thread of the kernel for few rows calls it.
__device__ __forceinline__ void allow_merge() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// CTAs of the attention kernel on a device of that many SMs; sets what divides by it.
template <int NT>
int ctas_for(ChunkLaunch &L, int sms)
{
    const int ctas = (sms < kSms ? sms : kSms) * (max_ctas<NT>() / kSms);
    L.ctas_mul = ~0ull / ctas + 1; // of no use, and not used, for one CTA
    return ctas;
}

template <int NT>
cudaError_t merge_launch(const ChunkLaunch &L, int ctas, cudaStream_t st)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, NT <= 64 ? NT / 4 : 16);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = NT <= 32 ? 1 : 0; // the kernel for many rows leaves it no registers
    return cudaLaunchKernelEx(&cfg, k_chunk_merge<NT>, L);
}

} // namespace chunk
} // namespace pw
