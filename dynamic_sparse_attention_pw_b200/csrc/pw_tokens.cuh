// pw_tokens.cuh -- device helpers shared by the kernels on new tokens.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "pw_internal.h"
#include "pw_sm100.cuh"
#include "pw_tokens.h"

namespace pw {
namespace tokens {

// Sequence of row t: the number of sequences that end at or before it (cu[i + 1] <= t), B if t
// lies behind the last one.  Called by a whole warp with a uniform t; each round looks at 32
// evenly spaced offsets, so a batch of up to 32 sequences takes one round of loads, one of up
// to 1024 two.  Any contents of cu give a result in [0, B].
__device__ __forceinline__ int find_sequence(const TokenBatch &tb, int64_t t, int lane)
{
    int lo = 0, n = tb.B; // the answer lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) >> 5;
        const int i = lo + (lane + 1) * step - 1; // this lane's sequence
        const bool before = i < lo + n && static_cast<int64_t>(__ldg(tb.cu + i + 1)) <= t;
        const int k = __popc(__ballot_sync(0xFFFFFFFFu, before));
        const int at = lo + k * step; // the first k of the looked-at sequences end before t
        n = min(step - 1, lo + n - at);
        lo = at;
    }
    return lo;
}

// Two f32 -> packed E4M3 pair (round to nearest even, magnitudes above 448 to 448, NaN kept);
// `lo` lands in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

using F2 = uint64_t; // two fp32, for the packed instructions

__device__ __forceinline__ F2 pack2(float lo, float hi)
{
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ void unpack2(F2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }

__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

} // namespace tokens
} // namespace pw
