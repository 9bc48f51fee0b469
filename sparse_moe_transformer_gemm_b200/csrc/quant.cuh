// quant.cuh -- e4m3 quantisation with a scale per block, shared by the kernels
// that quantise.
#pragma once

#include "common.cuh"

namespace moe {

// The quantisation of a block whose largest magnitude is `a`:
//   scale = a / 448 (1 where a = 0),  code = e4m3( 448 x / a ).
// Quotients come from a reciprocal and one residual correction (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990), which rounds as a division would. With bf16 x and a, 448 x is exact, and
// the quotient is a midpoint of two e4m3 values either exactly (five bits: the
// correction then yields it exactly) or by a distance of 2^-13 or more, so the
// code is the exact quotient's rounding. Very small and very large blocks are
// moved by a power of two first, so that nothing leaves the range of fp32.
struct BlockScale {
    float scale;   // what the codes are multiplied by
    float a, inv;  // the (moved) amax and its reciprocal
    float move;    // 448 times the power of two
};

__device__ __forceinline__ BlockScale block_scale(float a) {
    BlockScale b;
    const bool far = !(a >= 0x1p-60f && a <= 0x1p60f);  // (0, infinity and NaN too)
    const float p = !far ? 1.f : a < 1.f ? 0x1p100f : 0x1p-100f;
    b.a = a == 0.f ? 1.f : a * p;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b.a));  // b.a is in the normal range
    b.inv = fmaf(fmaf(-b.a, r, 1.f), r, r);
    b.move = 448.f * p;
    if (far) {
        b.scale = a == 0.f ? 1.f : a / 448.f;
    } else {
        const float q = a * (1.f / 448.f);
        b.scale = fmaf(fmaf(-q, 448.f, a), 1.f / 448.f, q);
    }
    return b;
}

__device__ __forceinline__ float block_quotient(const BlockScale& b, float x) {
    const float n = x * b.move;
    const float q = n * b.inv;
    return fmaf(fmaf(-q, b.a, n), b.inv, q);
}

// The same for two values, two at a time in each instruction.
struct BlockScale2 {
    uint64_t neg_a, inv, move;
};
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ BlockScale2 twice(const BlockScale& b) {
    return {pair_of(-b.a, -b.a), pair_of(b.inv, b.inv), pair_of(b.move, b.move)};
}
__device__ __forceinline__ float2 block_quotient2(const BlockScale2& b, float lo, float hi) {
    uint64_t n, q, r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(n) : "l"(pair_of(lo, hi)), "l"(b.move));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(n), "l"(b.inv));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q), "l"(b.neg_a), "l"(n));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(r), "l"(b.inv), "l"(q));
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
    return f;
}

// Two codes, the first in the low byte (values within 448 by construction).
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace moe
