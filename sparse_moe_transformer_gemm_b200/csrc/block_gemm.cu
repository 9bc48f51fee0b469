// block_gemm.cu -- FP8 (e4m3) matrix products with an fp32 scale per block of
// 128, dense or grouped by row offsets, and the SwiGLU gate_up form whose
// result is quantised again.
//
//   out[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{c in block b} xq[m, c] wq[n, c]
//   gate_up:  h = SiLU(g) u in fp32, hq / sh its quantisation per 128 features
//
// A thread owns one weight row and 16 tokens; the products of a block of 128
// columns are summed in fp32 and then scaled, since the scales differ per block.
#include "internal.h"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int NT = 16;  // tokens per tile

struct Args {
    const uint8_t* xq;
    const float* sx;
    const uint8_t* wq;
    const float* sw;
    const int* offsets;
    int G, M, N, K;
    void* out;
    float* out_scales;
};

// The 128 columns of block kb of weight row `w` times the NT staged tokens,
// added to acc with the blocks' scales.
__device__ __forceinline__ void block_dot(float (&acc)[NT], const uint8_t* w, int cols, float sw,
                                          const float (&xs)[NT][128], const float (&sxs)[NT]) {
    float part[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) part[t] = 0.f;
    for (int c = 0; c < cols; c += 16) {
        float f[16];
        e4m3x16_to_float(*reinterpret_cast<const uint4*>(w + c), f);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) part[t] = fmaf(f[i], xs[t][c + i], part[t]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = fmaf(part[t], sw * sxs[t], acc[t]);
}

template <bool GATE_UP, bool OUT_F32>
__global__ void __launch_bounds__(128)
block_gemm_kernel(const Args a) {
    pdl_launch_and_wait();
    __shared__ float xs[NT][128];
    __shared__ float sxs[NT];
    __shared__ uint32_t amax[4][NT];
    const int g = blockIdx.z, n = blockIdx.x * 128 + threadIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kb_n = (a.K + 127) / 128, nb_n = (a.N + 127) / 128;
    int r0 = 0, r1 = a.M;
    if (a.offsets) {
        r0 = min(max(a.offsets[g], 0), a.M);
        r1 = min(max(a.offsets[g + 1], 0), a.M);
    }
    const int rows_w = GATE_UP ? 2 * a.N : a.N;
    const uint8_t* w = a.wq + (size_t)g * rows_w * a.K;
    const float* sw = a.sw + (size_t)g * (GATE_UP ? 2 * nb_n : nb_n) * kb_n;
    for (int row0 = r0 + blockIdx.y * NT; row0 < r1; row0 += gridDim.y * NT) {
        float acc[NT], up[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = up[t] = 0.f;
        for (int kb = 0; kb < kb_n; ++kb) {
            const int cols = min(128, a.K - kb * 128);
            __syncthreads();
            for (int i = threadIdx.x; i < NT * 8; i += 128) {
                const int t = i >> 3, c = (i & 7) * 16;
                float f[16];
                if (row0 + t < r1 && c < cols) {
                    e4m3x16_to_float(*reinterpret_cast<const uint4*>(
                                         a.xq + (size_t)(row0 + t) * a.K + kb * 128 + c), f);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) xs[t][c + j] = f[j];
            }
            if (threadIdx.x < NT)
                sxs[threadIdx.x] = row0 + threadIdx.x < r1
                                       ? a.sx[(size_t)(row0 + threadIdx.x) * kb_n + kb] : 0.f;
            __syncthreads();
            if (n < a.N) {
                block_dot(acc, w + (size_t)n * a.K + kb * 128, cols,
                          sw[(size_t)blockIdx.x * kb_n + kb], xs, sxs);
                if constexpr (GATE_UP)
                    block_dot(up, w + (size_t)(a.N + n) * a.K + kb * 128, cols,
                              sw[(size_t)(nb_n + blockIdx.x) * kb_n + kb], xs, sxs);
            }
        }
        if constexpr (GATE_UP) {
            // N is a multiple of 128: the CTA holds one block of h per token
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                acc[t] = silu_mul(acc[t], up[t]);
                const uint32_t m = __reduce_max_sync(0xffffffffu, f32_bits(acc[t]) & 0x7FFFFFFFu);
                if (lane == 0) amax[warp][t] = m;
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const BlockScale b = block_scale(f32_from_bits(
                    max(max(amax[0][t], amax[1][t]), max(amax[2][t], amax[3][t]))));
                const uint32_t q = e4m3x2_of(block_quotient(b, acc[t]), 0.f);
                if (row0 + t < r1) {
                    static_cast<uint8_t*>(a.out)[(size_t)(row0 + t) * a.N + n] = (uint8_t)q;
                    if (threadIdx.x == 0)
                        a.out_scales[(size_t)(row0 + t) * nb_n + blockIdx.x] = b.scale;
                }
            }
        } else if (n < a.N) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (row0 + t < r1) {
                    const size_t at = (size_t)(row0 + t) * a.N + n;
                    if (OUT_F32)
                        static_cast<float*>(a.out)[at] = acc[t];
                    else
                        static_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(acc[t]);
                }
        }
    }
}

template <bool GATE_UP, bool OUT_F32>
cudaError_t launch(const BlockGemm& p, cudaStream_t s) {
    const Args a = {static_cast<const uint8_t*>(p.xq), p.sx, static_cast<const uint8_t*>(p.wq),
                    p.sw, p.offsets, p.G, p.M, p.N, p.K, p.out, p.out_scales};
    const int per_group = (p.M + p.G - 1) / p.G;
    const int y = (per_group + NT - 1) / NT;
    const dim3 grid((p.N + 127) / 128, y < 256 ? y : 256, p.G);
    const cudaError_t err = launch_pdl(block_gemm_kernel<GATE_UP, OUT_F32>, grid, dim3(128), 0, s, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_gemm(const BlockGemm& p, cudaStream_t s) {
    return p.out_type == MOE_OUT_F32 ? launch<false, true>(p, s) : launch<false, false>(p, s);
}
cudaError_t launch_block_gate_up(const BlockGemm& p, cudaStream_t s) {
    return launch<true, false>(p, s);
}

}  // namespace moe
