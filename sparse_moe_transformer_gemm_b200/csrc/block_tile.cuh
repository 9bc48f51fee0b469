// block_tile.cuh -- what the three block-FP8 product kernels share: the arguments,
// the table of tiles and the tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include <atomic>

#include "internal.h"
#include "quant.cuh"
#include "tc.cuh"

namespace moe {
namespace block {

constexpr int BK = 128;       // columns per scale block = bytes per staged row
constexpr int MAX_G = 257;    // 256 experts and a shared one
constexpr int NBOX = 16;      // rows of the smallest token box

struct Args {
    const float* sx;
    const float* sw;
    const int* offsets;
    int G, M, N, K;    // N: output features (gate_up: d_ff)
    int m_tiles;       // weight tiles of a group
    int w_rows;        // weight rows of a group (gate_up: 2 * d_ff)
    void* out;
    float* out_scales;
    int* status;
    const uint8_t* pf;   // weights to pull into L2 before the wait for the previous kernel
    long long pf_bytes;
};

// Token rows [M, K] bytes, boxes of 16, 32, 64 and 128 rows x 128 bytes.
struct TokenMaps {
    CUtensorMap m[4];
};

struct TileTable {
    int total;
    int off[MAX_G + 1];         // rows of group g: [off[g], off[g + 1])
    int tile_start[MAX_G + 1];  // its first tile
};

struct Tile {
    int g, m, row0, len;
};

// One warp fills the table: ceil(rows / NM) token tiles per weight tile. Offsets
// are clamped to [0, M], so that no bad value leads outside the buffers.
template <int NM>
__device__ __forceinline__ void fill_table(TileTable& c, const Args& a) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int b = 0; b <= a.G; b += 32) {
        const int g = b + lane;
        auto offset = [&](int i) {
            if (!a.offsets) return i == 0 ? 0 : a.M;
            return min(max(a.offsets[i], 0), a.M);
        };
        int cnt = 0;
        if (g <= a.G) {
            const int o = offset(g);
            c.off[g] = o;
            if (g < a.G) cnt = max(0, (offset(g + 1) - o + NM - 1) / NM) * a.m_tiles;
        }
        int incl = cnt;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, s);
            if (lane >= s) incl += v;
        }
        if (g < a.G) c.tile_start[g] = carry + incl - cnt;
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
        c.tile_start[a.G] = carry;
        c.total = carry;
    }
}

// Tile t: token tiles fastest (tiles that read the same weights are neighbours in
// time, so HBM gives them once and L2 the other times), then weight tiles, then
// groups.
template <int NM>
__device__ __forceinline__ Tile tile_of(const TileTable& c, int G, int t) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c.tile_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int rows = c.off[lo + 1] - c.off[lo];
    const int nt = (rows + NM - 1) / NM;
    const int local = t - c.tile_start[lo];
    const int m = local / nt, j = local - m * nt;
    return Tile{lo, m, c.off[lo] + j * NM, min(NM, rows - j * NM)};
}

// A pair's tiles pair, pair + n_pairs, ..., looked up once by the whole block (each
// role would spend 300 to 1000 cycles a tile on it); the ones past the list's end
// are looked up as they come.
constexpr int LIST = 256;
struct TileList {
    int4 t[LIST];
};
template <int NM>
__device__ __forceinline__ void fill_list(TileList& l, const TileTable& c, int G, int pair,
                                          int n_pairs) {
    for (int i = threadIdx.x; i < LIST; i += blockDim.x) {
        const int t = pair + i * n_pairs;
        if (t >= c.total) break;
        const Tile ti = tile_of<NM>(c, G, t);
        l.t[i] = make_int4(ti.g, ti.m, ti.row0, ti.len);
    }
}

// The tile in uniform registers (all lanes hold the same one).
__device__ __forceinline__ Tile uniform_tile(const Tile& t) {
    return Tile{(int)tc::uniform(t.g), (int)tc::uniform(t.m), (int)tc::uniform(t.row0),
                (int)tc::uniform(t.len)};
}

template <int NM>
__device__ __forceinline__ Tile listed_tile(const TileList& l, const TileTable& c, int G, int i,
                                            int t) {
    if (i >= LIST) return uniform_tile(tile_of<NM>(c, G, t));
    const int4 v = l.t[i];
    return uniform_tile(Tile{v.x, v.y, v.z, v.w});
}

// `rows` (a multiple of 16, at most 128) token rows from `row` on, as at most
// four boxes, completing on the even CTA's barrier.
__device__ __forceinline__ void load_tokens(uint8_t* dst, const TokenMaps& tm, uint32_t bar,
                                            int col, int row, int rows, uint64_t policy) {
    for (int o = 0; o < rows;) {
        const int rem = rows - o;
        const int lg = rem >= 128 ? 3 : rem >= 64 ? 2 : rem >= 32 ? 1 : 0;
        tc::tma_load_2d_pair(dst + o * BK, &tm.m[lg], bar, col, row + o, policy);
        o += NBOX << lg;
    }
}

// a += d * s on two fp32 values at a time.
__device__ __forceinline__ void fma2(uint64_t& a, uint64_t d, uint64_t s) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(d), "l"(s));
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
template <int N>
__device__ __forceinline__ float value_at(const uint64_t (&a)[N], int i) {
    return __uint_as_float((uint32_t)(a[i >> 1] >> (32 * (i & 1))));
}

// Host: maps and launch. make_byte_map: row-major [rows, cols] bytes, box of
// box_rows rows x 128 bytes, 128-byte swizzle.
bool make_byte_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                   uint32_t box_rows);
// make_token_byte_maps: the first `boxes` of them (16, 32, ... rows).
bool make_token_byte_maps(TokenMaps* tm, const void* base, uint64_t rows, uint64_t cols, int boxes);
int sm_pairs();

// A kernel's shared-memory limit, set once per device (`done`: a bit per device).
// cudaErrorLaunchOutOfResources: it was compiled to fewer registers than it hands over.
cudaError_t allow_smem(const void* kernel, int smem, std::atomic<uint64_t>& done,
                       const tc::RegSplit& split = {});

// The kernel on `pairs` pairs of SMs (allow_smem comes first).
template <typename Kernel>
cudaError_t launch_pairs(Kernel kernel, int pairs, int threads, int smem, cudaStream_t s,
                         const CUtensorMap& ma, const TokenMaps& mb, const Args& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_pdl
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, ma, mb, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// K slices of one product whose tiles of 128 weight rows (and up to 32 tokens, or 128) fit
// the SMs at once: the most, up to 8 (the portable cluster size) and the blocks of K,
// with which all clusters run at once; 0 for more tiles than SMs. A cluster's SMs lie
// in one GPC, and of its CTAs an SM holds one, so that a B200's 148 SMs take 15
// clusters of 8 and 33 of 4 (cudaOccupancyMaxActiveClusters on four GPUs), not 18 and 37.
// Constants, not the device's answer: a product has the same bits on every GPU.
// Measured at K = 4096, M = 1, with 8 / 4 / 2 slices: 15 tiles 5.0 / 5.7 / 7.8 us, 16 tiles
// 8.9 / 5.7 / 7.8, 33 tiles 13.6 / 6.1 / 7.9, 34 tiles 13.7 / 10.7 / 7.9, 74 tiles - / 16.4
// / 8.2 (uncut 12.1); M = 128: 15 tiles 8.1 / 8.8 / 11.9, 16 tiles 14.4 / 8.7 / 11.9, 33
// tiles 22.0 / 9.2 / 12.1, 34 tiles 22.2 / 16.5 / 12.1. Against the pair kernels: 128 x 4096
// x 4096 (32 tiles) 10.2 us and 31, 512 x 2048 x 4096 (64) 13.7 and 23, 512 x 4096 x 4096
// (128, uncut) 21.3 and 23.8, 200 x 256 x 128 (4, one block) 6.8 and 6.8.
__host__ __device__ constexpr int slices_of(long tiles, int blocks, int sms) {
    if (tiles > sms) return 0;
    int S = tiles <= 15 ? 8 : tiles <= 33 ? 4 : 2;
    while (S > 1 && (S * tiles > sms || S > blocks)) S /= 2;
    return S;
}

// The kernels' launchers (block_split.cu, block_few.cu, block_many.cu); splits: slices_of
// a product for block_split's kernel, 0 where it does not take it.
int splits(const BlockGemm& p);
cudaError_t launch_split(const BlockGemm& p, cudaStream_t s);
cudaError_t launch_few(const BlockGemm& p, bool gate_up, cudaStream_t s);
cudaError_t launch_many(const BlockGemm& p, bool gate_up, cudaStream_t s);

}  // namespace block
}  // namespace moe
