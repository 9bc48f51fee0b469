// quant.cuh -- e4m3 quantisation with a scale per block, shared by the kernels
// that quantise.
#pragma once

#include "common.cuh"

namespace moe {

// The quantisation of a block whose largest magnitude is `a`:
//   scale = a / 448 (1 where a = 0),  code = e4m3( 448 x / a ).
// The quotient is formed from the block's correctly rounded reciprocal with
// one residual correction (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990), which rounds it as a division
// would: with bf16 x and a, whose quotient times 448 is a midpoint of two
// e4m3 values either exactly or by a distance of 2^-13 or more, the code is
// the exact quotient's rounding. Very small and very large blocks are moved by
// a power of two first, so that neither 448 x nor the reciprocal leaves the
// range of fp32.
struct BlockScale {
    float scale;   // what the codes are multiplied by
    float a, inv;  // the (moved) amax and its reciprocal
    float move;    // 448 times the power of two
};

__device__ __forceinline__ BlockScale block_scale(float a) {
    BlockScale b;
    b.scale = a == 0.f ? 1.f : a / 448.f;
    const float p = a < 0x1p-60f ? 0x1p100f : a > 0x1p60f ? 0x1p-100f : 1.f;
    b.a = a == 0.f ? 1.f : a * p;
    b.inv = 1.f / b.a;
    b.move = 448.f * p;
    return b;
}

__device__ __forceinline__ float block_quotient(const BlockScale& b, float x) {
    const float n = x * b.move;
    const float q = n * b.inv;
    return fmaf(fmaf(-q, b.a, n), b.inv, q);
}

// Two codes, the first in the low byte (values within 448 by construction).
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace moe
