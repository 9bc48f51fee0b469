// block_split.cu -- a block-scaled FP8 product with few rows and few tiles (see
// block_gemm.cu): K is split over the CTAs of a cluster.
//
// A projection of a decode batch has N / 512 tiles of the pair kernels, 8 at N =
// 4096, for 74 pairs: its time is one tile's walk through K. Here a tile is 128
// weight rows (the MMA's M) times up to NT tokens (its N), on one SM, and S CTAs of
// a cluster take K / S of its columns each, so that N = 4096 has 32 S tiles. Each CTA
// adds its blocks to fp32 registers as block_few.cu does, leaves the partial sums
// in shared memory, and after a cluster barrier CTA r adds the S partial sums of the
// tokens r, r + S, ... in a fixed order, through distributed shared memory, a warp per
// token with 16 bytes a lane (by single floats 128 x 4096 x 4096 took 11.3 us).
//
// The bound is latency: the loads of the ring's first stages, the walk over K / S,
// the exchange. Measured: 1 x 4096 x 4096 in 6.5 us (the pair kernel: 13), 128 x
// 4096 x 4096 in 10 (31).
//
// Per CTA (384 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA issuer,
// warp 2 the factors sx[token] sw, warps 4-11 promotion in two groups of four (one
// warp per TMEM lane quarter). All waits are bounded.
#include "block_tile.cuh"

namespace moe {
namespace block {
namespace {

constexpr int BM = 128;
constexpr int SCALE_WARP = 2, PROMO_WARP = 4;
constexpr int GROUPS = 2;  // promotion groups of 4 warps
constexpr int THREADS = 32 * (PROMO_WARP + 4 * GROUPS);
constexpr int CH = 16;  // tokens per promotion chunk; group g takes the chunks g, g + 2, ...
constexpr int MAX_STAGES = 10;

template <int NT>
struct Shape {
    static constexpr int STAGE_BYTES = (BM + NT) * BK;  // 20 / 32 KB
    static constexpr int STAGES = NT == 32 ? 10 : 6;
    static constexpr int ACC = 512 / NT;  // blocks in flight in TMEM
    static constexpr int SLOTS = 8;       // factor ring
};

template <int NT>
struct Ctrl {
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t acc_full[Shape<NT>::ACC];
    uint64_t acc_empty[Shape<NT>::ACC];
    uint64_t sc_full[Shape<NT>::SLOTS];
    uint64_t sc_empty[Shape<NT>::SLOTS];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    alignas(16) float scales[Shape<NT>::SLOTS][NT];
};
template <int NT>
constexpr int smem_bytes() {
    return Shape<NT>::STAGES * Shape<NT>::STAGE_BYTES + 1024 + (int)sizeof(Ctrl<NT>);
}
static_assert(smem_bytes<32>() <= 232448 && smem_bytes<128>() <= 232448, "fits in 227 KB");
// the partial sums [NT][128] fp32 reuse the ring
static_assert(128 * BM * 4 <= Shape<128>::STAGES * Shape<128>::STAGE_BYTES, "partial sums fit");

// acc[token] += d[token] * s[token] (d: TMEM words, s: shared memory).
__device__ __forceinline__ void promote(uint64_t (&acc)[CH / 2], const uint32_t (&d)[CH],
                                        const float* s) {
#pragma unroll
    for (int j = 0; j < CH / 4; ++j) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s + 4 * j);
        fma2(acc[2 * j], pack2(d[4 * j], d[4 * j + 1]), f.x);
        fma2(acc[2 * j + 1], pack2(d[4 * j + 2], d[4 * j + 3]), f.y);
    }
}

// Token maps in use: tiles hold up to 16, 32 or 128 rows.
__host__ __device__ constexpr int boxes(int M, int NT) { return M <= 16 ? 1 : NT == 32 ? 2 : 4; }

// grid (row tiles, token tiles, S), clusters (1, 1, S). tmA: weights [N, K] bytes, box
// 128 x 128; tmB: tokens [M, K] bytes.
template <int NT, bool OUT_F32>
__global__ void __launch_bounds__(THREADS, 1)
block_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ TokenMaps tmB,
                   const Args a, int S) {
    using H = Shape<NT>;
    pdl_launch_and_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);  // stays a shared pointer
    Ctrl<NT>& c = *reinterpret_cast<Ctrl<NT>*>(smem + H::STAGES * H::STAGE_BYTES);
    const int warp = (int)tc::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int split = (int)tc::cluster_ctarank();
    const int KB = (a.K + BK - 1) / BK;
    const int kb0 = split * KB / S, kb1 = (split + 1) * KB / S;  // S <= KB: never empty
    const int row0 = blockIdx.y * NT, len = min(NT, a.M - row0);
    const int n = (len + 15) & ~15;  // the MMA's N
    const int w0 = blockIdx.x * BM;  // first weight row

    if (warp == 0) {
        if (lane == 0) {
            c.abort = 0;
            tc::prefetch_tensormap(&tmA);
            for (int m = 0; m < boxes(a.M, NT); ++m) tc::prefetch_tensormap(&tmB.m[m]);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < H::STAGES; ++s) {
                tc::mbar_init(&c.full[s], 1);
                tc::mbar_init(&c.empty[s], 1);
            }
            for (int i = 0; i < H::ACC; ++i) {
                tc::mbar_init(&c.acc_full[i], 1);
                tc::mbar_init(&c.acc_empty[i], 4 * GROUPS);
            }
            for (int i = 0; i < H::SLOTS; ++i) {
                tc::mbar_init(&c.sc_full[i], 1);
                tc::mbar_init(&c.sc_empty[i], 4 * GROUPS);
            }
            tc::mbar_init(&c.drain, 1);
            tc::fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc(&c.tmem_base, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem_base = tc::uniform(c.tmem_base);
    const volatile int* abort_flag = &c.abort;
    auto give_up = [&]() {
        *reinterpret_cast<volatile int*>(&c.abort) = 1;
        atomicExch(a.status, MOE_ERR_TIMEOUT);
    };

    float* part = reinterpret_cast<float*>(smem);  // [NT][128], once the ring is idle
    constexpr int NCH = NT / CH / GROUPS;  // chunks of a group
    uint64_t acc[NCH][CH / 2];
    const int grp = (warp - PROMO_WARP) >> 2;
    bool ok = true;
    if (warp == 0) {
        // ---------------- producer
        const uint64_t pol_w = tc::policy_evict_first();
        const uint64_t pol_x = tc::policy_evict_last();
        uint32_t it = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const uint32_t stage = it % H::STAGES;
            if (!tc::mbar_wait_warp(&c.empty[stage], ((it / H::STAGES) & 1u) ^ 1u, abort_flag)) {
                give_up();
                break;
            }
            uint8_t* s = smem + stage * H::STAGE_BYTES;
            if (tc::elect_one()) {
                tc::mbar_arrive_expect_tx(&c.full[stage], (uint32_t)(BM + n) * BK);
                tc::tma_load_2d_hint(s, &tmA, &c.full[stage], kb * BK, w0, pol_w);
                for (int o = 0; o < n;) {
                    const int rem = n - o;
                    const int lg = rem >= 128 ? 3 : rem >= 64 ? 2 : rem >= 32 ? 1 : 0;
                    tc::tma_load_2d_hint(s + (BM + o) * BK, &tmB.m[lg], &c.full[stage], kb * BK,
                                         row0 + o, pol_x);
                    o += NBOX << lg;
                }
            }
            __syncwarp();
        }
        // every copy has landed before the CTA's shared memory is used for other things
        const int zero = 0;
        for (uint32_t i = it < H::STAGES ? 0 : it - H::STAGES; i < it; ++i)
            if (!tc::mbar_wait(&c.full[i % H::STAGES], (i / H::STAGES) & 1u, &zero))
                atomicExch(a.status, MOE_ERR_TIMEOUT);
    } else if (warp == 1) {
        // ---------------- MMA issuer: 128 weight rows x n tokens
        const uint32_t idesc = tc::idesc_e4m3_f32(BM, n);
        uint32_t blk = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++blk) {
            const uint32_t as = blk % H::ACC, stage = blk % H::STAGES;
            if (!tc::mbar_wait_warp(&c.acc_empty[as], ((blk / H::ACC) & 1u) ^ 1u, abort_flag) ||
                !tc::mbar_wait_warp(&c.full[stage], (blk / H::STAGES) & 1u, abort_flag)) {
                give_up();
                break;
            }
            tc::fence_after_sync();
            const uint32_t w = tc::smem_u32(smem + stage * H::STAGE_BYTES);
            if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < BK / 32; ++k)
                    tc::mma_e4m3(tmem_base + as * NT, tc::desc_sw128(w + k * 32),
                                 tc::desc_sw128(w + BM * BK + k * 32), idesc, k > 0);
                tc::mma_commit(&c.empty[stage]);
                tc::mma_commit(&c.acc_full[as]);
            }
            __syncwarp();
        }
        if (tc::elect_one()) tc::mma_commit(&c.drain);
        __syncwarp();
        const int zero = 0;
        if (!tc::mbar_wait(&c.drain, 0, &zero)) atomicExch(a.status, MOE_ERR_TIMEOUT);
    } else if (warp == SCALE_WARP) {
        // ---------------- factors, U blocks loaded at a time
        constexpr int TPL = NT / 32, U = NT == 32 ? 4 : 2;
        const float* sxp = a.sx + (size_t)(row0 + lane) * KB;
        const float* swp = a.sw + (size_t)blockIdx.x * KB;
        uint32_t blk = 0;
        for (int k0 = kb0; k0 < kb1 && ok; k0 += U) {
            float x[TPL][U], w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = k0 + u < kb1 ? swp[k0 + u] : 0.f;
#pragma unroll
                for (int i = 0; i < TPL; ++i)
                    x[i][u] = k0 + u < kb1 && lane + 32 * i < len
                                  ? sxp[(size_t)(32 * i) * KB + k0 + u] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k0 + u >= kb1 || !ok) continue;
                const uint32_t slot = blk % H::SLOTS;
                ok = tc::mbar_wait_warp(&c.sc_empty[slot], ((blk / H::SLOTS) & 1u) ^ 1u, abort_flag);
                if (!ok) {
                    give_up();
                    continue;
                }
#pragma unroll
                for (int i = 0; i < TPL; ++i) c.scales[slot][lane + 32 * i] = x[i][u] * w[u];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&c.sc_full[slot]);
                ++blk;
            }
        }
    } else if (warp >= PROMO_WARP) {
        // ---------------- promotion: lane = one weight row, half of the tokens
        const uint32_t lane_base = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int j = 0; j < CH / 2; ++j) acc[i][j] = 0;
        uint32_t blk = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++blk) {
            const uint32_t as = blk % H::ACC, slot = blk % H::SLOTS;
            ok = tc::mbar_wait_warp(&c.sc_full[slot], (blk / H::SLOTS) & 1u, abort_flag) &&
                 tc::mbar_wait_warp(&c.acc_full[as], (blk / H::ACC) & 1u, abort_flag);
            if (!ok) {
                give_up();
                break;
            }
            tc::fence_after_sync();
            // two chunks at a time
#pragma unroll
            for (int i = 0; i < NCH; i += 2) {
                const int t0 = (GROUPS * i + grp) * CH, t1 = t0 + GROUPS * CH;
                if (t0 >= n) continue;
                const bool both = i + 1 < NCH && t1 < n;
                uint32_t d0[CH], d1[CH];
                tc::tmem_ld16(lane_base + as * NT + t0, d0);
                if (both) tc::tmem_ld16(lane_base + as * NT + t1, d1);
                tc::tmem_ld_wait();
                tc::tmem_loaded(d0);
                if (both) tc::tmem_loaded(d1);
                promote(acc[i], d0, c.scales[slot] + t0);
                if (both) promote(acc[i + 1 < NCH ? i + 1 : i], d1, c.scales[slot] + t1);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&c.acc_empty[as]);
                tc::mbar_arrive(&c.sc_empty[slot]);
            }
        }
    }

    // the ring is idle: every load has landed and every MMA has read its operands
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const int row = (threadIdx.x - 32 * PROMO_WARP) & 127;
    if (warp >= PROMO_WARP) {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int t = (GROUPS * i + grp) * CH + j;
                if (t < len) part[t * BM + row] = value_at(acc[i], j);
            }
    }
    tc::cluster_sync();
    {
        // a warp takes one token at a time, of CTA split's every S-th, a lane 4 weight rows of
        // it; the S partial sums in the order of the slices
        const uint32_t base = tc::smem_u32(part);
        uint32_t from[8];
#pragma unroll
        for (int sp = 0; sp < 8; ++sp) from[sp] = tc::map_to_cta(base, sp < S ? sp : 0);
        const int r4 = lane * 4, valid = a.N - (w0 + r4);  // valid rows of this lane
        for (int t = split + warp * S; t < len; t += THREADS / 32 * S) {
            const uint32_t off = (uint32_t)(t * BM + r4) * 4u;
            float4 v[8];
#pragma unroll
            for (int sp = 0; sp < 8; ++sp)
                if (sp < S) v[sp] = tc::ld_cluster_f32x4(from[sp] + off);
            float4 sum = v[0];
#pragma unroll
            for (int sp = 1; sp < 8; ++sp)
                if (sp < S) {
                    sum.x += v[sp].x;
                    sum.y += v[sp].y;
                    sum.z += v[sp].z;
                    sum.w += v[sp].w;
                }
            if (valid <= 0) continue;
            const size_t at = (size_t)(row0 + t) * a.N + w0 + r4;
            const float f[4] = {sum.x, sum.y, sum.z, sum.w};
            if constexpr (OUT_F32) {
                float* o = static_cast<float*>(a.out) + at;
                if (a.N % 4 == 0)
                    *reinterpret_cast<float4*>(o) = sum;
                else
                    for (int j = 0; j < 4; ++j)
                        if (j < valid) o[j] = f[j];
            } else {
                uint16_t* o = static_cast<uint16_t*>(a.out) + at;
                if (a.N % 4 == 0) {
                    uint16_t h[4];
                    for (int j = 0; j < 4; ++j) h[j] = float_to_bf16_bits(f[j]);
                    *reinterpret_cast<uint2*>(o) =
                        make_uint2(h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
                } else {
                    for (int j = 0; j < 4; ++j)
                        if (j < valid) o[j] = float_to_bf16_bits(f[j]);
                }
            }
        }
    }
    tc::cluster_sync();  // nobody leaves while its partial sums are read
    if (warp == 1) {
        __syncwarp();
        tc::tmem_dealloc(tmem_base, 512);
    }
}

template <int NT, bool OUT_F32>
cudaError_t launch(const BlockGemm& p, int S, cudaStream_t s) {
    const Args a = {p.sx, p.sw, nullptr, 1, p.M, p.N, p.K, 0, p.N, p.out, nullptr, p.status,
                    nullptr, 0};
    CUtensorMap ma;
    TokenMaps mb;
    if (!make_byte_map(&ma, p.wq, p.N, p.K, BM) ||
        !make_token_byte_maps(&mb, p.xq, p.M, p.K, boxes(p.M, NT)))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    auto kernel = block_split_kernel<NT, OUT_F32>;
    cudaError_t err = allow_smem((const void*)kernel, smem_bytes<NT>(), done);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.N + BM - 1) / BM, (p.M + NT - 1) / NT, S);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<NT>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = S;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_pdl
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kernel, ma, mb, a, S);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

int splits(const BlockGemm& p) {
    if (p.offsets) return 0;
    const long token_tiles = p.M <= 32 ? 1 : (p.M + 127) / 128;
    return slices_of((p.N + BM - 1) / BM * token_tiles, (p.K + BK - 1) / BK, 2 * sm_pairs());
}

cudaError_t launch_split(const BlockGemm& p, cudaStream_t s) {
    const int S = splits(p);
    if (p.M <= 32)
        return p.out_type == MOE_OUT_F32 ? launch<32, true>(p, S, s) : launch<32, false>(p, S, s);
    return p.out_type == MOE_OUT_F32 ? launch<128, true>(p, S, s) : launch<128, false>(p, S, s);
}

}  // namespace block
}  // namespace moe
