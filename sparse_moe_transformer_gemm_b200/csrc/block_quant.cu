// block_quant.cu -- quantise bf16 activation rows to e4m3 with one fp32 scale
// per 128 columns (moe_block_quant), and the same on the way to the grouped
// rows of the experts (moe_block_permute: each token is read and quantised once
// and its codes are written to its k rows).
//
// Eight lanes take one block of 128 columns, twice 16 bytes a lane: the largest
// magnitude is an integer maximum on the bf16 patterns without their signs
// (which also orders infinities and NaN above every finite value), so one pass
// reads x once and writes the codes once.
//
// Bound: HBM, 2 M K bytes read and M K (1 + 1/32) written; 16384 x 4096 in 33 us (6.2
// TB/s), 40 with cold caches. With half as many columns a lane, and so twice the
// shuffles and divisions a value, the instructions were the bound: 44 us.
#include "internal.h"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int WARPS = 4;
constexpr int CHUNK = 512;  // columns of a warp's unit: four blocks
constexpr int CTAS_PER_SM = 10;

// Two pieces of 8 columns of one row (their bf16 patterns; zero where the row has
// ended) to 8 code bytes each; the 8 lanes of the block share its scale.
__device__ __forceinline__ uint32_t max2(const uint4& u) {
    return __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                    __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
}
__device__ __forceinline__ uint2 codes_of(const BlockScale2& b2, const uint4& u) {
    auto pair = [&](uint32_t v) {
        const float2 x = bf16x2_to_float2(v);
        const float2 q = block_quotient2(b2, x.x, x.y);
        return e4m3x2_of(q.x, q.y);
    };
    return make_uint2(pair(u.x) | (pair(u.y) << 16), pair(u.z) | (pair(u.w) << 16));
}
__device__ __forceinline__ float quantise16(const uint4 (&u)[2], uint2 (&q)[2]) {
    uint32_t m = __vmaxu2(max2(u[0]), max2(u[1]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale b = block_scale(f32_from_bits(max(m >> 16, m & 0xFFFFu) << 16));
    const BlockScale2 b2 = twice(b);
    q[0] = codes_of(b2, u[0]);
    q[1] = codes_of(b2, u[1]);
    return b.scale;
}

// A unit is 512 columns of one row. The warps take the units in turn, U at a time
// (2 KB on the way per warp), whatever the rows' length: row and chunk of a unit
// follow from the last one's by an addition. PERMUTE: row t goes to the kk rows
// row_of[t * kk + j] of the output (entries outside [0, R) are skipped).
template <bool PERMUTE>
__global__ void __launch_bounds__(WARPS * 32, CTAS_PER_SM)
block_quant_kernel(const __nv_bfloat16* __restrict__ x, long ldx, int M, int K,
                   const int* __restrict__ row_of, int kk, long R, uint8_t* __restrict__ codes,
                   float* __restrict__ scales, int* clear) {
    pdl_launch_and_wait();
    if (PERMUTE && clear && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0;
    constexpr int U = 2;
    const int lane = threadIdx.x & 31;
    const int kb = (K + 127) / 128, chunks = (K + CHUNK - 1) / CHUNK;
    const int warps = gridDim.x * WARPS, w = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const int d_row = warps / chunks, d_chunk = warps - d_row * chunks;
    int row = w / chunks, chunk = w - row * chunks;
    while (row < M) {
        uint4 u[U][2];
        int r0[U], c0[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            r0[i] = row;
            c0[i] = chunk * CHUNK + (lane >> 3) * 128 + (lane & 7) * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                u[i][h] = row < M && c0[i] + 64 * h < K
                              ? ld_stream_u4(x + row * ldx + c0[i] + 64 * h)
                              : make_uint4(0, 0, 0, 0);
            row += d_row;
            chunk += d_chunk;
            if (chunk >= chunks) {
                chunk -= chunks;
                ++row;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (r0[i] >= M) break;  // uniform
            uint2 q[2];
            const float scale = quantise16(u[i], q);
            const int c = c0[i];
            if (c >= K) continue;
            auto store = [&](long r) {
                uint8_t* o = codes + r * K + c;
                *reinterpret_cast<uint2*>(o) = q[0];
                if (c + 64 < K) *reinterpret_cast<uint2*>(o + 64) = q[1];
                if ((lane & 7) == 0) scales[r * kb + (c >> 7)] = scale;
            };
            if constexpr (PERMUTE) {
                for (int j = 0; j < kk; ++j) {
                    const long r = row_of[(long)r0[i] * kk + j];
                    if (r >= 0 && r < R) store(r);
                }
            } else {
                store(r0[i]);
            }
        }
    }
}

unsigned grid_of(int M, int K) {
    const long units = (long)M * ((K + CHUNK - 1) / CHUNK);
    const long ctas = (units + WARPS - 1) / WARPS, most = 148L * CTAS_PER_SM;
    return (unsigned)(ctas < most ? ctas : most);
}

}  // namespace

cudaError_t launch_block_quant(const void* x, long ldx, int M, int K, void* codes, float* scales,
                               cudaStream_t s) {
    const cudaError_t err = launch_pdl(
        block_quant_kernel<false>, dim3(grid_of(M, K)), dim3(WARPS * 32), 0, s,
        static_cast<const __nv_bfloat16*>(x), ldx, M, K, (const int*)nullptr, 1, 0L,
        static_cast<uint8_t*>(codes), scales, (int*)nullptr);
    return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_block_permute(const void* x, const int32_t* row_of, int T, int kk, int d,
                                 long R, void* codes, float* scales, int* clear, cudaStream_t s) {
    const cudaError_t err = launch_pdl(
        block_quant_kernel<true>, dim3(grid_of(T, d)), dim3(WARPS * 32), 0, s,
        static_cast<const __nv_bfloat16*>(x), (long)d, T, d, row_of, kk, R,
        static_cast<uint8_t*>(codes), scales, clear);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe
