// block_few.cu -- block-scaled FP8 products for few rows a group (see
// block_gemm.cu), on pairs of SMs (tcgen05 cta_group::2, kind::f8f6f4).
//
// The weight stream is the bound: every weight byte is read once and used for a
// handful of tokens. The weight rows are the MMA's M (256 a pair and
// accumulator, 128 a CTA) and up to NM = 32, 64 or 128 tokens its N, so a tile
// costs the tensor core little; two accumulators share the staged tokens
// (gate_up: gate and up rows, whose SiLU(g) u is then formed in registers; a
// plain product: two 256-row tiles). A block's sums take 2 NM TMEM columns, so 8,
// 4 or 2 blocks are in flight between the MMAs and the promotion, and the ring
// holds 6, 5 or 4 stages of 32 KB of weights per SM.
//
// NM = 32 for up to a row a group on average, 64 for up to 32 rows, 128 beyond: a
// group in one tile has its weights read once, a smaller tile keeps more blocks in
// flight and is done sooner. The experts d = 4096, d_ff = 1536, E = 192, top-8,
// whole layer, tokens evenly over the experts / expert e's share falling as e^-0.5:
//              32           64            128
//   T = 1      50           51            53
//   T = 64     503 / 456    505 / 456     508 / 465
//   T = 256    547 / 557    548 / 548     552 / 552
//   T = 512    578 / 616    579 / 597     587 / 598
//   T = 1024   725 / 742    616 / 681     625 / 668
//   T = 2048   1038 / 1121  1020 / 918    743 / 855 us
// At T = 64 the layer reads 3.4 GB: 6.7 TB/s.
//
// A thread of the promotion owns one weight row and NM / 2 tokens of each
// accumulator. A CTA's 128 weight rows of an accumulator lie in one block of
// rows, so the factor sx[token] sw[rows] of a token is the same for the whole
// CTA: a warp forms them in a ring in shared memory, ahead of the promotion.
//
// Per CTA (384 threads): warp 0 TMA producer, warp 1 TMEM owner (+ MMA issuer in
// the even CTA), warp 2 the factors, warps 4-11 promotion and epilogue in two
// groups of four (one warp per TMEM lane quarter) with NM / 2 tokens each. All
// waits are bounded.
#include "block_tile.cuh"

namespace moe {
namespace block {
namespace {

constexpr int BM = 128;                // weight rows per CTA and accumulator
constexpr int A_BYTES = BM * BK;
constexpr int CH = 16;                 // tokens per promotion chunk
constexpr int SLOTS = 8;               // factor ring
// Blocks a CTA loads ahead of the MMAs where a pair has several tiles: enough to cover
// the latency; with more of them in flight HBM serves all of them more slowly. The
// layer of the header with 4 and with the whole ring (6 or 5): T = 64 503 and 519 us,
// T = 256 546 and 559, T = 512 577 and 597, T = 1024 612 and 650; 3: 508, 560, 594, 640.
// One token, whose 8 experts give a pair one tile or none, takes 51.0 with 4, 49.9 with 6.
constexpr uint32_t AHEAD = 4;
constexpr int SCALE_WARP = 2, PROMO_WARP = 4;
constexpr int THREADS = 32 * (PROMO_WARP + 8);
// Registers a thread with tiles of 128 tokens, whose promotion holds 128
// accumulators: 168 at launch; 3 * 168 = 72 + 2 * 216.
constexpr int REGS_FEW = 72, REGS_MANY = 216;
constexpr tc::RegSplit REGS = {REGS_FEW, REGS_MANY, 2};
static_assert(tc::split_fits(REGS, 168) && !tc::split_fits(REGS, 160), "all of a launch with 168");
// Up to so many rows a group on average, tiles of 64 tokens.
constexpr long kFewRows64 = 32;

// NM: tokens per pair tile at most.
template <int NM>
struct Shape {
    static constexpr int STAGE_BYTES = 2 * A_BYTES + NM / 2 * BK;  // 34 / 36 / 40 KB
    static constexpr int STAGES = NM == 32 ? 6 : NM == 64 ? 5 : 4;  // what fits
    static_assert(STAGES >= (int)AHEAD);
    static constexpr int COLS = 2 * NM;     // TMEM columns per block
    static constexpr int ACC = 512 / COLS;  // blocks in flight
    static constexpr int NCH = NM / 2 / CH; // chunks of a group and accumulator
    // per group: gate_up a [NM / 2 tokens][128 features] tile of codes, else a [16
    // tokens][128 rows] tile of bf16
    static constexpr int EPI_BYTES = 2 * (NM / 2 * BM > CH * BM * 2 ? NM / 2 * BM : CH * BM * 2);
};

constexpr int boxes(int NM) { return NM == 32 ? 1 : NM == 64 ? 2 : 3; }  // token maps in use

template <int NM>
struct Ctrl {
    uint64_t full[Shape<NM>::STAGES];    // even CTA: TMA bytes of both CTAs landed
    uint64_t empty[Shape<NM>::STAGES];   // both CTAs: the pair MMAs finished reading the stage
    uint64_t acc_full[Shape<NM>::ACC];   // both CTAs: a block's sums are in TMEM
    uint64_t acc_empty[Shape<NM>::ACC];  // even CTA: every promotion warp has read them
    uint64_t sc_full[SLOTS];
    uint64_t sc_empty[SLOTS];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    TileTable tab;
    alignas(16) TileList list;
    alignas(16) float scales[SLOTS][Shape<NM>::COLS];
    alignas(16) float4 hscale[2][NM / 2];  // gate_up: BlockScale of a token
};
template <int NM>
constexpr int smem_bytes() {
    return Shape<NM>::STAGES * Shape<NM>::STAGE_BYTES + Shape<NM>::EPI_BYTES + 1024 +
           (int)sizeof(Ctrl<NM>);
}
static_assert(smem_bytes<32>() <= 232448 && smem_bytes<64>() <= 232448 &&
                  smem_bytes<128>() <= 232448, "fits in 227 KB");

template <int NM>
__device__ __forceinline__ void give_up(Ctrl<NM>& c, int* status) {
    *reinterpret_cast<volatile int*>(&c.abort) = 1;
    atomicExch(status, MOE_ERR_TIMEOUT);
}

// acc[token] += d[token] * s[token] (d: TMEM words, s: shared memory).
__device__ __forceinline__ void promote(uint64_t (&acc)[CH / 2], const uint32_t (&d)[CH],
                                        const float* s) {
#pragma unroll
    for (int i = 0; i < CH / 4; ++i) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s + 4 * i);
        fma2(acc[2 * i], pack2(d[4 * i], d[4 * i + 1]), f.x);
        fma2(acc[2 * i + 1], pack2(d[4 * i + 2], d[4 * i + 3]), f.y);
    }
}

// tmA: weights [G * w_rows, K] bytes, box 128 x 128; tmB: tokens [M, K] bytes.
template <bool GATE_UP, bool OUT_F32, int NM>
__global__ void __launch_bounds__(THREADS, 1)
block_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ TokenMaps tmB,
                 const Args a) {
    using S = Shape<NM>;
    constexpr int STAGES = S::STAGES, ACC = S::ACC, COLS = S::COLS, NCH = S::NCH;
    constexpr int R = NCH >= 2 ? 2 : 1;  // chunks per load round
    pdl_launch();
    // The weights are read-only in the layer: while the routing and the grouping still
    // run, the blocks that are resident already pull the first experts' weights into
    // L2, a slice each in 64 KB requests.
    if (a.pf_bytes > 0 && threadIdx.x == 0) {
        const long long per = ((a.pf_bytes + gridDim.x - 1) / gridDim.x + 15) & ~15ll;
        const long long b0 = (long long)blockIdx.x * per;
        const long long b1 = b0 + per < a.pf_bytes ? b0 + per : a.pf_bytes;
        for (long long o = b0; o < b1; o += 65536)
            tc::prefetch_l2_bulk(a.pf + o, (uint32_t)(b1 - o < 65536 ? b1 - o : 65536));
    }
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);  // stays a shared pointer
    uint8_t* epi = smem + STAGES * S::STAGE_BYTES;
    Ctrl<NM>& c = *reinterpret_cast<Ctrl<NM>*>(epi + S::EPI_BYTES);
    const int warp = (int)tc::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = (int)(tc::cluster_ctarank() & 1u);
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    const int KB = (a.K + BK - 1) / BK;

    // ---- prologue: tile table (warp 0), barriers and TMEM (warp 1), in both CTAs
    if (warp == 0) {
        fill_table<NM>(c.tab, a);
        if (lane == 0) {
            c.abort = 0;
            tc::prefetch_tensormap(&tmA);
            for (int m = 0; m < boxes(NM); ++m) tc::prefetch_tensormap(&tmB.m[m]);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < STAGES; ++s) {
                tc::mbar_init(&c.full[s], 1);
                tc::mbar_init(&c.empty[s], 1);
            }
            for (int i = 0; i < ACC; ++i) {
                tc::mbar_init(&c.acc_full[i], 1);
                tc::mbar_init(&c.acc_empty[i], 2 * 8);
            }
            for (int i = 0; i < SLOTS; ++i) {
                tc::mbar_init(&c.sc_full[i], 1);
                tc::mbar_init(&c.sc_empty[i], 8);
            }
            tc::mbar_init(&c.drain, 1);
            tc::fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc_pair(&c.tmem_base, 512);
        tc::tmem_relinquish_pair();
    }
    tc::fence_before_sync();
    tc::cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
    tc::fence_after_sync();
    fill_list<NM>(c.list, c.tab, a.G, pair, n_pairs);
    __syncthreads();
    const uint32_t tmem_base = tc::uniform(c.tmem_base);
    const int total = (int)tc::uniform(c.tab.total);
    const volatile int* abort_flag = &c.abort;
    // first weight row of a tile's accumulator p, within its group, for this CTA
    auto first_row = [&](int m, int p) {
        return GATE_UP ? p * a.N + m * 2 * BM + rank * BM : m * 4 * BM + p * 2 * BM + rank * BM;
    };
    // the MMA's N: 32, or the tile's tokens rounded up to 32
    auto tokens_of = [&](const Tile& ti) { return NM == 32 ? 32 : (ti.len + 31) & ~31; };
    // whether the pair's accumulator 1 has rows (always in gate_up)
    auto two = [&](int m) { return GATE_UP || m * 4 * BM + 2 * BM < a.N; };

    if (warp >= PROMO_WARP) {
        if constexpr (NM == 128) tc::regs_inc<REGS_MANY>();
        // ---------------- promotion and epilogue: lane = one weight row of each
        // accumulator; group grp takes the tokens [grp * half, (grp + 1) * half), half of
        // the MMA's N, in chunks of 16
        const int quad = warp & 3, grp = (warp - PROMO_WARP) >> 2;
        const int et = threadIdx.x - 32 * PROMO_WARP - 128 * grp;  // 0..127 within the group
        const int bar = 1 + grp;
        const int row = quad * 32 + lane;                          // of the CTA's 128
        const uint32_t lane_base = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint32_t acc_empty0 = tc::map_to_cta(tc::smem_u32(&c.acc_empty[0]), 0);
        uint8_t* tile = epi + grp * (S::EPI_BYTES / 2);
        uint32_t blk = 0;
        for (int t = pair, i_t = 0; t < total; t += n_pairs, ++i_t) {
            const Tile ti = listed_tile<NM>(c.list, c.tab, a.G, i_t, t);
            const int half = tokens_of(ti) / 2, col0 = grp * half;
            const int left = min(half, ti.len - col0);  // valid tokens of this group
            const long tok0 = ti.row0 + col0;
            const bool second = two(ti.m);
            uint64_t acc[2][NCH][CH / 2];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < NCH; ++i)
#pragma unroll
                    for (int j = 0; j < CH / 2; ++j) acc[p][i][j] = 0;
            bool ok = true;
            for (int kb = 0; kb < KB; ++kb, ++blk) {
                uint32_t as = blk % ACC, slot = blk % SLOTS;
                // (in vector registers: the uniform path takes longer, T = 2048 740 us for 728)
                tc::opaque(as);
                tc::opaque(slot);
                ok = tc::mbar_wait_warp(&c.sc_full[slot], (blk / SLOTS) & 1u, abort_flag) &&
                     tc::mbar_wait_warp(&c.acc_full[as], (blk / ACC) & 1u, abort_flag);
                if (!ok) break;
                if (left > 0) {
                    tc::fence_after_sync();
                    const uint32_t tb = lane_base + as * COLS + col0;
                    const float* sc = c.scales[slot] + col0;
#pragma unroll
                    for (int i = 0; i < NCH; i += R) {
                        if (i * CH >= left) continue;
                        uint32_t d0[R][CH], d1[R][CH];
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            if (r > 0 && (i + r) * CH >= left) continue;
                            tc::tmem_ld16(tb + (i + r) * CH, d0[r]);
                            if (second) tc::tmem_ld16(tb + NM + (i + r) * CH, d1[r]);
                        }
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            tc::tmem_loaded(d0[r]);
                            tc::tmem_loaded(d1[r]);
                        }
                        if ((i + R) * CH >= left) {  // the last chunks: the block is read
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive_cluster_read(acc_empty0 + as * 8);
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            if (r > 0 && (i + r) * CH >= left) continue;
                            promote(acc[0][i + r], d0[r], sc + (i + r) * CH);
                            if (second) promote(acc[1][i + r], d1[r], sc + NM + (i + r) * CH);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&c.sc_empty[slot]);
                } else if (lane == 0) {
                    tc::mbar_arrive_cluster_read(acc_empty0 + as * 8);
                    tc::mbar_arrive(&c.sc_empty[slot]);
                }
            }
            // a warp that gave up takes its group with it
            if (tc::bar_any(bar, 128, !ok)) {
                give_up(c, a.status);
                break;
            }
            if (left <= 0) continue;
            if constexpr (GATE_UP) {
                const int f0 = ti.m * 2 * BM + rank * BM;  // first feature of the CTA's block
                // a token's largest |h| of each lane quarter, in the tile's space
                uint32_t (*amax)[4] = reinterpret_cast<uint32_t(*)[4]>(tile);
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    if (i * CH >= left) continue;
                    uint32_t mx = 0;
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        const float h0 = silu_mul(value_at(acc[0][i], j), value_at(acc[1][i], j));
                        const float h1 =
                            silu_mul(value_at(acc[0][i], j + 1), value_at(acc[1][i], j + 1));
                        acc[0][i][j / 2] = pack2(f32_bits(h0), f32_bits(h1));
                        const uint32_t m0 =
                            __reduce_max_sync(0xffffffffu, f32_bits(h0) & 0x7FFFFFFFu);
                        const uint32_t m1 =
                            __reduce_max_sync(0xffffffffu, f32_bits(h1) & 0x7FFFFFFFu);
                        if (lane == j) mx = m0;
                        if (lane == j + 1) mx = m1;
                    }
                    if (lane < CH) amax[i * CH + lane][quad] = mx;
                }
                tc::bar_sync(bar, 128);
                if (et < left) {
                    const uint4 m = *reinterpret_cast<const uint4*>(amax[et]);
                    const BlockScale b =
                        block_scale(f32_from_bits(max(max(m.x, m.y), max(m.z, m.w))));
                    c.hscale[grp][et] = make_float4(b.a, b.inv, b.move, b.scale);
                    if (f0 < a.N) a.out_scales[(tok0 + et) * (a.N / 128) + (f0 >> 7)] = b.scale;
                }
                tc::bar_sync(bar, 128);
                // codes through a [tokens][128 features] tile to 16-byte stores
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    if (i * CH >= left) continue;
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const float4 v = c.hscale[grp][i * CH + j];
                        const BlockScale b = {v.w, v.x, v.y, v.z};
                        tile[(i * CH + j) * BM + row] =
                            (uint8_t)e4m3x2_of(block_quotient(b, value_at(acc[0][i], j)), 0.f);
                    }
                }
                tc::bar_sync(bar, 128);
                if (f0 < a.N)
                    for (int id = et; id < left * (BM / 16); id += 128) {
                        const int n = id / (BM / 16), ch = id % (BM / 16);
                        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + (tok0 + n) * a.N +
                                                  f0 + ch * 16) =
                            *reinterpret_cast<const uint4*>(tile + n * BM + ch * 16);
                    }
                // (the next tile's bar_any comes before the next writes here)
            } else {
                const bool vec = !OUT_F32 && a.N % 8 == 0;
                uint16_t* o = reinterpret_cast<uint16_t*>(tile);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int n0 = first_row(ti.m, p);  // first output column
                    if (p == 1 && !second) continue;
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        if (i * CH >= left) continue;
                        if (vec) {
                            // through a [16 tokens][128 rows] tile to 16-byte stores
                            if (p + i > 0) tc::bar_sync(bar, 128);  // the last one is read
#pragma unroll
                            for (int j = 0; j < CH; ++j)
                                o[j * BM + row] = float_to_bf16_bits(value_at(acc[p][i], j));
                            tc::bar_sync(bar, 128);
#pragma unroll
                            for (int q = 0; q < CH * BM / 8 / 128; ++q) {
                                const int id = et + 128 * q;
                                const int n = id / (BM / 8), ch = id % (BM / 8);
                                if (i * CH + n < left && n0 + ch * 8 < a.N)
                                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                              (tok0 + i * CH + n) * a.N + n0 +
                                                              ch * 8) =
                                        *reinterpret_cast<const uint4*>(o + n * BM + ch * 8);
                            }
                        } else if (n0 + row < a.N) {
#pragma unroll
                            for (int j = 0; j < CH; ++j)
                                if (i * CH + j < left) {
                                    const long at = (tok0 + i * CH + j) * a.N + n0 + row;
                                    if (OUT_F32)
                                        static_cast<float*>(a.out)[at] = value_at(acc[p][i], j);
                                    else
                                        static_cast<uint16_t*>(a.out)[at] =
                                            float_to_bf16_bits(value_at(acc[p][i], j));
                                }
                        }
                    }
                }
            }
        }
    } else {
        if constexpr (NM == 128) tc::regs_dec<REGS_FEW>();
        if (warp == 0) {
            // ---------------- producer: this CTA's weight rows and half of the tokens
            const uint64_t pol_w = tc::policy_evict_first();
            const uint64_t pol_x = tc::policy_evict_last();
            const uint32_t ahead = total > n_pairs ? AHEAD : STAGES;
            uint32_t it = 0;  // blocks loaded
            bool ok = true;
            for (int t = pair, i_t = 0; t < total && ok; t += n_pairs, ++i_t) {
                const Tile ti = listed_tile<NM>(c.list, c.tab, a.G, i_t, t);
                const bool second = two(ti.m);
                const int w0 = ti.g * a.w_rows + first_row(ti.m, 0);
                const int w1 = ti.g * a.w_rows + first_row(ti.m, 1);
                const int half = tokens_of(ti) / 2;
                const uint32_t bytes = 2u * ((second ? 2 : 1) * A_BYTES + half * BK);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const uint32_t stage = it % STAGES;
                    // (blocks are released in order: the one before the last that may be in
                    // flight is read, so the one that had this stage is too)
                    const uint32_t old = it - ahead;
                    if (it >= ahead &&
                        !tc::mbar_wait_warp(&c.empty[old % STAGES], (old / STAGES) & 1u, abort_flag)) {
                        give_up(c, a.status);
                        ok = false;
                        break;
                    }
                    const uint32_t bar = tc::map_to_cta(tc::smem_u32(&c.full[stage]), 0);
                    uint8_t* s = smem + stage * S::STAGE_BYTES;
                    if (tc::elect_one()) {
                        if (leader) tc::mbar_arrive_expect_tx(&c.full[stage], bytes);
                        tc::tma_load_2d_pair(s, &tmA, bar, kb * BK, w0, pol_w);
                        if (second) tc::tma_load_2d_pair(s + A_BYTES, &tmA, bar, kb * BK, w1, pol_w);
                        if (NM == 32)
                            tc::tma_load_2d_pair(s + 2 * A_BYTES, &tmB.m[0], bar, kb * BK,
                                                 ti.row0 + rank * CH, pol_x);
                        else
                            load_tokens(s + 2 * A_BYTES, tmB, bar, kb * BK, ti.row0 + rank * half,
                                        half, pol_x);
                    }
                    __syncwarp();
                }
            }
            // drain: this CTA's copies have landed (the even CTA's full barrier saw
            // every byte of both CTAs when its last phase completed)
            const int zero = 0;
            for (uint32_t i = it < STAGES ? 0 : it - STAGES; i < it; ++i) {
                const uint32_t stage = i % STAGES;
                if (!tc::mbar_wait(leader ? &c.full[stage] : &c.empty[stage], (i / STAGES) & 1u, &zero))
                    atomicExch(a.status, MOE_ERR_TIMEOUT);
            }
        } else if (warp == 1) {
            if (leader) {
                // ---------------- MMA issuer (even CTA): 256 weight rows x n tokens, twice
                uint32_t blk = 0;
                bool ok = true;
                for (int t = pair, i_t = 0; t < total && ok; t += n_pairs, ++i_t) {
                    const Tile ti = listed_tile<NM>(c.list, c.tab, a.G, i_t, t);
                    const bool second = two(ti.m);
                    const uint32_t idesc = tc::idesc_e4m3_f32(2 * BM, tokens_of(ti));
                    for (int kb = 0; kb < KB; ++kb, ++blk) {
                        const uint32_t as = blk % ACC, stage = blk % STAGES;
                        if (!tc::mbar_wait_warp(&c.acc_empty[as], ((blk / ACC) & 1u) ^ 1u, abort_flag) ||
                            !tc::mbar_wait_warp(&c.full[stage], (blk / STAGES) & 1u, abort_flag)) {
                            give_up(c, a.status);
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t d = tmem_base + as * COLS;
                        const uint32_t w = tc::smem_u32(smem + stage * S::STAGE_BYTES);
                        if (tc::elect_one()) {
#pragma unroll
                            for (int k = 0; k < BK / 32; ++k) {
                                const uint64_t x = tc::desc_sw128(w + 2 * A_BYTES + k * 32);
                                tc::mma_e4m3_pair(d, tc::desc_sw128(w + k * 32), x, idesc, k > 0);
                                if (second)
                                    tc::mma_e4m3_pair(d + NM, tc::desc_sw128(w + A_BYTES + k * 32), x,
                                                      idesc, k > 0);
                            }
                            tc::mma_commit_pair(&c.empty[stage], 0x3);
                            tc::mma_commit_pair(&c.acc_full[as], 0x3);
                        }
                        __syncwarp();
                    }
                }
                if (tc::elect_one()) tc::mma_commit_pair(&c.drain, 0x1);
                __syncwarp();
                const int zero = 0;
                if (!tc::mbar_wait(&c.drain, 0, &zero)) atomicExch(a.status, MOE_ERR_TIMEOUT);
            }
        } else if (warp == SCALE_WARP) {
            // ---------------- factors: per block sx[token] * sw of this CTA's weight rows, U
            // blocks loaded at a time. The ring runs ahead of the promotion, over tile
            // borders too.
            constexpr int U = NM == 128 ? 2 : 4, TPL = NM / 32;  // tokens per lane
            const int nb_n = (a.N + 127) / 128;
            const int sw_rows = GATE_UP ? 2 * nb_n : nb_n;
            uint32_t blk = 0;
            bool ok = true;
            for (int t = pair, i_t = 0; t < total && ok; t += n_pairs, ++i_t) {
                const Tile ti = listed_tile<NM>(c.list, c.tab, a.G, i_t, t);
                const float* sxp = a.sx + (size_t)(ti.row0 + lane) * KB;
                const float* swp[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int nb = min(first_row(ti.m, p) / BM, sw_rows - 1);
                    swp[p] = a.sw + ((size_t)ti.g * sw_rows + nb) * KB;
                }
                for (int k0 = 0; k0 < KB && ok; k0 += U) {
                    float x[TPL][U], w[2][U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool in = k0 + u < KB;
                        w[0][u] = in ? swp[0][k0 + u] : 0.f;
                        w[1][u] = in ? swp[1][k0 + u] : 0.f;
#pragma unroll
                        for (int i = 0; i < TPL; ++i)
                            x[i][u] = in && lane + 32 * i < ti.len
                                          ? sxp[(size_t)(32 * i) * KB + k0 + u] : 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (k0 + u >= KB || !ok) continue;
                        const uint32_t slot = blk % SLOTS;
                        ok = tc::mbar_wait_warp(&c.sc_empty[slot], ((blk / SLOTS) & 1u) ^ 1u, abort_flag);
                        if (!ok) {
                            give_up(c, a.status);
                            continue;
                        }
#pragma unroll
                        for (int i = 0; i < TPL; ++i) {
                            c.scales[slot][lane + 32 * i] = x[i][u] * w[0][u];
                            c.scales[slot][NM + lane + 32 * i] = x[i][u] * w[1][u];
                        }
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&c.sc_full[slot]);
                        ++blk;
                    }
                }
            }
        }
    }

    // Neither CTA leaves while the other may still signal its barriers or read
    // its shared memory.
    tc::fence_before_sync();
    tc::cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem_base, 512);
    }
}

template <bool GATE_UP, bool OUT_F32, int NM>
cudaError_t launch(const CUtensorMap& ma, const TokenMaps& mb, const Args& a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    auto kernel = block_few_kernel<GATE_UP, OUT_F32, NM>;
    const cudaError_t err = allow_smem((const void*)kernel, smem_bytes<NM>(), done,
                                       NM == 128 ? REGS : tc::RegSplit{});
    return err != cudaSuccess
               ? err
               : launch_pairs(kernel, sm_pairs(), THREADS, smem_bytes<NM>(), s, ma, mb, a);
}

// Bytes of weights gate_up pulls into L2 ahead, where nearly every expert has rows (two
// a group on average: 86% of them); else what is pulled may be another expert's.
// Measured, Hy3 experts: T = 256 574 -> 567 us, T = 64 (a shorter grouping) 515 -> 514;
// the same for down, whose blocks become resident late, changed nothing.
constexpr long long kPrefetch = 48ll << 20;
long long prefetched(const BlockGemm& p, bool gate_up, long long bytes) {
    if (!gate_up || !p.offsets || p.M < 2L * p.G) return 0;
    return (bytes < kPrefetch ? bytes : kPrefetch) & ~15ll;
}

template <int NM>
cudaError_t launch_nm(const BlockGemm& p, bool gate_up, cudaStream_t s) {
    const int w_rows = gate_up ? 2 * p.N : p.N;
    const int per_tile = gate_up ? 2 * BM : 4 * BM;
    const Args a = {p.sx, p.sw, p.offsets, p.G, p.M, p.N, p.K, (p.N + per_tile - 1) / per_tile,
                    w_rows, p.out, p.out_scales, p.status, static_cast<const uint8_t*>(p.wq),
                    prefetched(p, gate_up, (long long)p.G * w_rows * p.K)};
    CUtensorMap ma;
    TokenMaps mb;
    if (!make_byte_map(&ma, p.wq, (uint64_t)p.G * w_rows, p.K, BM) ||
        !make_token_byte_maps(&mb, p.xq, p.M, p.K, boxes(NM)))
        return cudaErrorInvalidValue;
    if (gate_up) return launch<true, false, NM>(ma, mb, a, s);
    if (p.out_type == MOE_OUT_F32) return launch<false, true, NM>(ma, mb, a, s);
    return launch<false, false, NM>(ma, mb, a, s);
}

}  // namespace

cudaError_t launch_few(const BlockGemm& p, bool gate_up, cudaStream_t s) {
    if (p.M <= p.G || (!p.offsets && p.M <= 32)) return launch_nm<32>(p, gate_up, s);
    if ((long)p.M <= kFewRows64 * p.G) return launch_nm<64>(p, gate_up, s);
    return launch_nm<128>(p, gate_up, s);
}

}  // namespace block
}  // namespace moe
