// block_quant.cu -- quantise bf16 activation rows to e4m3 with one fp32 scale
// per 128 columns (moe_block_quant), and the same on the way to the grouped
// rows of the experts (moe_block_permute: each token is read and quantised once
// and its codes are written to its k rows).
//
// A half-warp takes one block of 128 columns, 16 bytes a lane: the largest
// magnitude is an integer maximum on the bf16 patterns without their signs
// (which also orders infinities and NaN above every finite value), so one pass
// reads x once and writes the codes once.
//
// Bound: HBM, 2 M K bytes read and M K (1 + 1/32) written.
#include "internal.h"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int WARPS = 4;
constexpr int CHUNK = 256;  // columns of a warp's pass: two blocks

// The 8 columns [col, col + 8) of one row (u: their bf16 patterns; zero where
// the row has ended) to 8 code bytes; the 16 lanes of the block share its scale.
__device__ __forceinline__ uint2 quantise8(const uint4& u, float& scale) {
    uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                          __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t top = max(m >> 16, m & 0xFFFFu);
    const BlockScale b = block_scale(f32_from_bits(top << 16));
    scale = b.scale;
    float f[8];
    bf16x8_to_float(u, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = block_quotient(b, f[i]);
    return make_uint2(e4m3x2_of(f[0], f[1]) | (e4m3x2_of(f[2], f[3]) << 16),
                      e4m3x2_of(f[4], f[5]) | (e4m3x2_of(f[6], f[7]) << 16));
}

// WPR warps share a row (a power of two <= WARPS), each taking every WPR-th
// chunk. PERMUTE: row t goes to the kk rows row_of[t * kk + j] of the output
// (entries outside [0, R) are skipped).
template <bool PERMUTE>
__global__ void __launch_bounds__(WARPS * 32)
block_quant_kernel(const __nv_bfloat16* __restrict__ x, long ldx, int M, int K, int wpr,
                   const int* __restrict__ row_of, int kk, long R, uint8_t* __restrict__ codes,
                   float* __restrict__ scales) {
    pdl_launch_and_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long row = (long)blockIdx.x * (WARPS / wpr) + warp / wpr;
    if (row >= M) return;
    const int kb = (K + 127) / 128;
    const __nv_bfloat16* src = x + row * ldx;
    constexpr int U = 4;  // chunks in flight
    for (int c0 = (warp % wpr) * CHUNK; c0 < K; c0 += U * wpr * CHUNK) {
        uint4 u[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int col = c0 + i * wpr * CHUNK + lane * 8;
            u[i] = col < K ? ld_stream_u4(src + col) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int col = c0 + i * wpr * CHUNK + lane * 8;
            float scale;
            const uint2 q = quantise8(u[i], scale);
            if (col >= K) continue;
            if constexpr (PERMUTE) {
                for (int j = 0; j < kk; ++j) {
                    const long r = row_of[row * kk + j];
                    if (r < 0 || r >= R) continue;
                    *reinterpret_cast<uint2*>(codes + r * K + col) = q;
                    if ((lane & 15) == 0) scales[r * kb + (col >> 7)] = scale;
                }
            } else {
                *reinterpret_cast<uint2*>(codes + row * K + col) = q;
                if ((lane & 15) == 0) scales[row * kb + (col >> 7)] = scale;
            }
        }
    }
}

int warps_per_row(int K) {
    const int chunks = (K + CHUNK - 1) / CHUNK;
    return chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
}

}  // namespace

cudaError_t launch_block_quant(const void* x, long ldx, int M, int K, void* codes, float* scales,
                               cudaStream_t s) {
    const int wpr = warps_per_row(K), rows = WARPS / wpr;
    const cudaError_t err =
        launch_pdl(block_quant_kernel<false>, dim3((unsigned)((M + rows - 1) / rows)),
                   dim3(WARPS * 32), 0, s, static_cast<const __nv_bfloat16*>(x), ldx, M, K, wpr,
                   (const int*)nullptr, 1, 0L, static_cast<uint8_t*>(codes), scales);
    return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_block_permute(const void* x, const int32_t* row_of, int T, int kk, int d,
                                 long R, void* codes, float* scales, cudaStream_t s) {
    const int wpr = warps_per_row(d), rows = WARPS / wpr;
    const cudaError_t err =
        launch_pdl(block_quant_kernel<true>, dim3((unsigned)((T + rows - 1) / rows)),
                   dim3(WARPS * 32), 0, s, static_cast<const __nv_bfloat16*>(x), (long)d, T, d, wpr,
                   row_of, kk, R, static_cast<uint8_t*>(codes), scales);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe
