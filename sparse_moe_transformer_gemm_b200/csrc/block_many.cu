// block_many.cu -- block-scaled FP8 products for many rows a group (see
// block_gemm.cu), on pairs of SMs (tcgen05 cta_group::2, kind::f8f6f4).
//
// A pair tile is 256 tokens (the MMA's M, 128 a CTA) times 256 weight rows (its N,
// each CTA staging 128 of them): 32 KB through shared memory per CTA and block
// of 128 columns. A block's sums start from zero in one of two 256-column TMEM
// accumulators, each handed over in two halves of 128 columns. A thread of the
// promotion owns one token and a half's 128 columns: the block's factor
// sx[token] sw[rows] is one register for 64 of them, and the sum of a block is one
// fused multiply-add per value. (With the weight rows in M and the tokens in N the
// factors differ per column and come from shared memory, 16 bytes per 4 values and
// thread: the product 8192 x 8192 x 4096 took 706 us that way.)
//
// gate_up: the even CTA stages the gate rows of one 128-feature block, the odd
// CTA its up rows; a half holds 64 features' gate columns, then their up columns.
// A thread holds 64 gate and the same 64 up values of its token, so SiLU(g) u, the
// token's largest |h| and the codes need no exchange but one float from each of
// the token's two threads.
//
// What bounds it: the promotion's chain of a block (waits, two rounds of tcgen05.ld,
// 128 two-value multiply-adds per scheduler), about 1000 cycles against 512 of MMAs;
// when the accumulators are handed back within it makes no difference. Without the
// loads from TMEM and the multiply-adds the product takes 170 us, without the multiply-adds
// 192, without the loads from L2 240. Measured steps, product 8192 x 8192 x 4096:
// factors loaded by the promotion itself 509 us, from a ring in shared memory 360 us;
// issuing warps with warp-uniform control flow (the MMA warp alone had needed 1000
// cycles a block), the factors waited for once in 4 blocks and four promotion groups in
// place of two 346 us; halves with an issuing warp each 305 us; a tile looked up once
// and waits as one short loop 282 us; the loop's state in vector registers, the factors
// loaded before the wait for the accumulator, warps without tokens not told apart 252
// us; two groups again, whose loads and multiply-adds overlap, 245 us (2.25 PFLOP/s),
// which also spills nothing and draws less power. 128 weight rows a tile with four
// accumulators in flight: 507 us. The next block's first loads under this one's last
// multiply-adds: 254 us.
//
// Per CTA (384 threads): warp 0 TMA producer, warps 1 and 3 (even CTA) MMA issuers of
// one half each, warp 1 also TMEM owner, warp 2 the factors (a ring in shared
// memory), warps 4-11 promotion and epilogue in a group per half (one warp per 32 TMEM
// lanes). The promotion's threads hold 192 values, so the first four warps hand
// registers over (setmaxnreg). All waits are bounded.
#include <type_traits>

#include "block_tile.cuh"

namespace moe {
namespace block {
namespace {

constexpr int BM = 128;                // tokens, and weight rows, a CTA stages
constexpr int NM = 2 * BM;             // tokens per pair tile
constexpr int STAGE_BYTES = 2 * BM * BK;
// 6 would fit. Fewer blocks in flight are served faster by HBM: the experts d = 4096,
// d_ff = 1536, E = 192, top-8 at T = 4096 take 1190 us with 5 and 1209 with 6, at T =
// 8192 2354 and 2398; with 4 1182 and 2340, but 2048 x 8192 x 4096 takes 90 us for 85.
constexpr int STAGES = 5;
constexpr int COLS = 256;              // TMEM columns per block
constexpr int GROUPS = 2;              // promotion groups of 4 warps, one per half
constexpr int PROMO_WARP = 4;          // the first of 8
constexpr int THREADS = 32 * (PROMO_WARP + 4 * GROUPS);
constexpr int CH = 32;                 // columns per tcgen05.ld
constexpr int SCALE_WARP = 2;
constexpr int FB = 4;                  // blocks per slot of the factor ring
constexpr int SLOTS = 2;
constexpr int EPI_BYTES = 4 * GROUPS * 32 * 32;  // a [32 tokens][32 bytes] store tile per warp
// registers a thread: 168 at launch; 3 * 168 = 72 + 2 * 216
constexpr int REGS_FEW = 72, REGS_MANY = 216;
constexpr tc::RegSplit REGS = {REGS_FEW, REGS_MANY, GROUPS};
static_assert(tc::split_fits(REGS, 168) && !tc::split_fits(REGS, 160), "all of a launch with 168");

struct Ctrl {
    uint64_t full[STAGES];    // even CTA: TMA bytes of both CTAs landed
    uint64_t empty[STAGES];   // both CTAs: the pair MMAs finished reading the stage
    // of each half of the columns:
    uint64_t acc_full[2][2];   // both CTAs: a block's sums are in TMEM
    uint64_t acc_empty[2][2];  // even CTA: the promotion warps of both CTAs have read them
    uint64_t sc_full[SLOTS];
    uint64_t sc_empty[SLOTS];
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
    TileTable tab;
    alignas(16) TileList list;
    float amax[GROUPS][BM];   // gate_up: a token's largest |h| in each group's columns
    float factor[SLOTS][FB][2][BM];  // sx[token] * sw of the columns 0-127 and 128-255
};
constexpr int SMEM = STAGES * STAGE_BYTES + EPI_BYTES + 1024 + (int)sizeof(Ctrl);
static_assert(SMEM <= 232448, "fits in 227 KB");

__device__ __forceinline__ void give_up(Ctrl& c, int* status) {
    *reinterpret_cast<volatile int*>(&c.abort) = 1;
    atomicExch(status, MOE_ERR_TIMEOUT);
}

__device__ __forceinline__ void promote(uint64_t (&acc)[CH / 2], const uint32_t (&d)[CH], float f) {
    const uint64_t ff = pack2(f32_bits(f), f32_bits(f));
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) fma2(acc[i], pack2(d[2 * i], d[2 * i + 1]), ff);
}

// tmA: weights [G * w_rows, K] bytes, box 128 x 128; tmB: tokens [M, K] bytes.
template <bool GATE_UP, bool OUT_F32>
__global__ void __launch_bounds__(THREADS, 1)
block_many_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ TokenMaps tmB,
                  const Args a) {
    pdl_launch_and_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);  // stays a shared pointer
    uint8_t* epi = smem + STAGES * STAGE_BYTES;
    Ctrl& c = *reinterpret_cast<Ctrl*>(epi + EPI_BYTES);
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
            for (int m = 0; m < 4; ++m) tc::prefetch_tensormap(&tmB.m[m]);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < STAGES; ++s) {
                tc::mbar_init(&c.full[s], 1);
                tc::mbar_init(&c.empty[s], 2);
            }
            for (int i = 0; i < 2; ++i) {
                for (int h = 0; h < 2; ++h) {
                    tc::mbar_init(&c.acc_full[i][h], 1);
                    tc::mbar_init(&c.acc_empty[i][h], 2 * 4);
                }
            }
            for (int i = 0; i < SLOTS; ++i) {
                tc::mbar_init(&c.sc_full[i], 1);
                tc::mbar_init(&c.sc_empty[i], 4 * GROUPS);
            }
            for (int h = 0; h < 2; ++h) tc::mbar_init(&c.drain[h], 1);
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

    if (warp >= PROMO_WARP) {
        tc::regs_inc<REGS_MANY>();
        // ---------------- promotion and epilogue: lane = one token of this CTA's
        // and the 128 columns of one half: 64 of the even CTA's weight rows, 64 of the odd's
        const int quad = warp & 3, half = (warp - PROMO_WARP) >> 2;
        const int row = quad * 32 + lane;
        const int nb_n = (a.N + 127) / 128;
        const uint32_t tcol = tmem_base + ((uint32_t)(quad * 32) << 16) + half * 128;
        const uint32_t acc_full0 = tc::smem_u32(&c.acc_full[0][half]);
        const uint32_t acc_empty0 = tc::map_to_cta(tc::smem_u32(&c.acc_empty[0][half]), 0);
        const uint32_t sc_full0 = tc::smem_u32(&c.sc_full[0]);
        const uint32_t sc_empty0 = tc::smem_u32(&c.sc_empty[0]);
        const uint32_t fac0 = tc::smem_u32(&c.factor[0][0][0][row]);
        // The loop's state in bytes, and in vector registers: kept as block counts the
        // compiler puts it and all that follows from it on the uniform path, 40
        // instructions a block and warp more and 7% of the kernel's time.
        constexpr uint32_t SLOT_BYTES = sizeof(c.factor[0]);
        uint32_t buf = 0, par = 0;        // 16 x the accumulator, its phase
        uint32_t fac_at = 0, sc_par = 0;  // the block's place in the ring of factors, its phase
        for (int t = pair, i_t = 0; t < total; t += n_pairs, ++i_t) {
            const Tile ti = listed_tile<NM>(c.list, c.tab, a.G, i_t, t);
            const int tok = rank * BM + row;  // token within the tile
            const bool mine = tok < ti.len;
            uint64_t acc[4][CH / 2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < CH / 2; ++j) acc[i][j] = 0;
            bool ok = true;
            for (int kb = 0; kb < KB; ++kb) {
                if (fac_at % SLOT_BYTES == 0)
                    ok = tc::mbar_wait_warp_at(sc_full0 + fac_at / SLOT_BYTES * 8, sc_par, abort_flag);
                const float f0 = tc::ld_shared_f32(fac0 + fac_at);
                const float f1 = tc::ld_shared_f32(fac0 + 4 * BM + fac_at);
                ok = tc::mbar_wait_warp_at(acc_full0 + buf, par, abort_flag) && ok;
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t tb = tcol + buf * (COLS / 16);
                uint32_t d0[CH], d1[CH];
                tc::tmem_ld32(tb, d0);
                tc::tmem_ld32(tb + CH, d1);
                tc::tmem_ld_wait();
                tc::tmem_loaded(d0);
                tc::tmem_loaded(d1);
                promote(acc[0], d0, f0);
                tc::tmem_ld32(tb + 2 * CH, d0);
                promote(acc[1], d1, f0);
                tc::tmem_ld32(tb + 3 * CH, d1);
                tc::tmem_ld_wait();
                tc::tmem_loaded(d0);
                tc::tmem_loaded(d1);
                tc::fence_before_sync();
                if (tc::elect_one()) tc::mbar_arrive_cluster_read(acc_empty0 + buf);
                __syncwarp();
                par ^= buf >> 4;
                buf ^= 16;
                fac_at += 2 * BM * 4;
                if (fac_at % SLOT_BYTES == 0 || kb + 1 == KB) {
                    if (lane == 0) tc::mbar_arrive_at(sc_empty0 + (fac_at - 1) / SLOT_BYTES * 8);
                    fac_at = (fac_at + SLOT_BYTES - 1) / SLOT_BYTES % SLOTS * SLOT_BYTES;
                    sc_par ^= fac_at == 0;
                }
                tc::opaque(buf);
                tc::opaque(par);
                tc::opaque(fac_at);
                tc::opaque(sc_par);
                promote(acc[2], d0, f1);
                promote(acc[3], d1, f1);
            }
            if constexpr (GATE_UP) {
                // h in acc[0] and acc[1]; the token's largest |h| over both groups' columns
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        const float h0 = silu_mul(value_at(acc[i], j), value_at(acc[i + 2], j));
                        const float h1 =
                            silu_mul(value_at(acc[i], j + 1), value_at(acc[i + 2], j + 1));
                        acc[i][j / 2] = pack2(f32_bits(h0), f32_bits(h1));
                        mx = max(mx, max(f32_bits(h0) & 0x7FFFFFFFu, f32_bits(h1) & 0x7FFFFFFFu));
                    }
                c.amax[half][row] = f32_from_bits(mx);
                // (a warp that gave up takes the others with it)
                if (tc::bar_any(1, 128 * GROUPS, !ok)) {
                    give_up(c, a.status);
                    break;
                }
                const BlockScale b = block_scale(f32_from_bits(
                    max(f32_bits(c.amax[0][row]), f32_bits(c.amax[1][row]))));
                const BlockScale2 b2 = twice(b);
                if (mine) {
                    const long r = ti.row0 + tok;
                    if (half == 0) a.out_scales[r * nb_n + ti.m] = b.scale;
                    uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + r * a.N +
                                                        ti.m * 128 + half * 2 * CH);
#pragma unroll
                    for (int q = 0; q < 2 * CH / 16; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const int j = (q & 1) * 16 + v * 4;
                            const auto& h = acc[q >> 1];
                            const float2 q0 =
                                block_quotient2(b2, value_at(h, j), value_at(h, j + 1));
                            const float2 q1 =
                                block_quotient2(b2, value_at(h, j + 2), value_at(h, j + 3));
                            w[v] = e4m3x2_of(q0.x, q0.y) | (e4m3x2_of(q1.x, q1.y) << 16);
                        }
                        o[q] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                tc::bar_sync(1, 128 * GROUPS);  // amax is read before the next tile's
            } else {
                if (!ok) {
                    give_up(c, a.status);
                    break;
                }
                if (rank * BM + quad * 32 >= ti.len) continue;  // no token of this warp
                const int rows = ti.len - rank * BM - quad * 32;  // tokens of this warp
                const long r0 = ti.row0 + rank * BM + quad * 32;
                // EC columns at a time through the warp's [32 tokens][32 bytes] tile, its
                // 16-byte halves swapped for every other four tokens (no bank conflicts):
                // whole 32-byte sectors go out, two lanes a row
                using Out = typename std::conditional<OUT_F32, float, uint16_t>::type;
                constexpr int EC = 32 / sizeof(Out), PIECE = 16 / sizeof(Out);
                const bool vec = a.N % PIECE == 0;
                uint4* st = reinterpret_cast<uint4*>(
                    epi + (warp - PROMO_WARP) * (EPI_BYTES / (4 * GROUPS)));
#pragma unroll
                for (int i = 0; i < 4 * CH / EC; ++i) {
                    // first output column: 64 of the even CTA's rows, then of the odd one's
                    const int n0 = ti.m * COLS + half * 64 + i * EC / 64 * 128 + i * EC % 64;
                    __syncwarp();  // the previous pass is read
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const auto& v = acc[i / (CH / EC)];
                        const int j = (i % (CH / EC)) * EC + q * PIECE;
                        uint4 u;
                        if constexpr (OUT_F32)
                            u = make_uint4(f32_bits(value_at(v, j)), f32_bits(value_at(v, j + 1)),
                                           f32_bits(value_at(v, j + 2)),
                                           f32_bits(value_at(v, j + 3)));
                        else
                            u = make_uint4(pack_bf16x2(value_at(v, j), value_at(v, j + 1)),
                                           pack_bf16x2(value_at(v, j + 2), value_at(v, j + 3)),
                                           pack_bf16x2(value_at(v, j + 4), value_at(v, j + 5)),
                                           pack_bf16x2(value_at(v, j + 6), value_at(v, j + 7)));
                        st[lane * 2 + (q ^ ((lane >> 2) & 1))] = u;
                    }
                    __syncwarp();
                    Out* o = static_cast<Out*>(a.out) + r0 * a.N + n0;
                    if (vec) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int n = q * 16 + (lane >> 1), ch = lane & 1;
                            if (n < rows && n0 + ch * PIECE < a.N)
                                *reinterpret_cast<uint4*>(o + (long)n * a.N + ch * PIECE) =
                                    st[n * 2 + (ch ^ ((n >> 2) & 1))];
                        }
                    } else {
                        // rows that are not 16-byte aligned: by elements, still in order
#pragma unroll 1
                        for (int e = lane; e < 32 * EC; e += 32) {
                            const int n = e / EC, c0 = e % EC, ch = c0 / PIECE;
                            if (n < rows && n0 + c0 < a.N)
                                o[(long)n * a.N + c0] = reinterpret_cast<const Out*>(
                                    st + n * 2 + (ch ^ ((n >> 2) & 1)))[c0 % PIECE];
                        }
                    }
                }
            }
        }
    } else {
        tc::regs_dec<REGS_FEW>();
        if (warp == 0) {
            // ---------------- producer: this CTA's 128 tokens and 128 weight rows
            const uint64_t pol_w = tc::policy_evict_first();
            const uint64_t pol_x = tc::policy_evict_last();
            uint32_t it = 0;  // blocks loaded
            bool ok = true;
            for (int t = pair, i_t = 0; t < total && ok; t += n_pairs, ++i_t) {
                const Tile ti = listed_tile<NM>(c.list, c.tab, a.G, i_t, t);
                // the rows that exist, in 16-row boxes; the others, which only reach TMEM
                // lanes that nobody reads, as zeros from past the end of the array (left as
                // they were they cost power: experts T = 8192 2770 us against 2735 after a
                // second of load, 2370 and 2360 before)
                const int rows = (min(max(ti.len - rank * BM, 0), BM) + 15) & ~15;
                constexpr uint32_t bytes = 2 * STAGE_BYTES;
                const int w0 = ti.g * a.w_rows +
                               (GATE_UP ? ti.m * BM + rank * a.N : ti.m * COLS + rank * BM);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const uint32_t stage = it % STAGES;
                    if (!tc::mbar_wait_warp(&c.empty[stage], ((it / STAGES) & 1u) ^ 1u,
                                            abort_flag)) {
                        give_up(c, a.status);
                        ok = false;
                        break;
                    }
                    const uint32_t bar = tc::map_to_cta(tc::smem_u32(&c.full[stage]), 0);
                    uint8_t* s = smem + stage * STAGE_BYTES;
                    if (tc::elect_one()) {
                        if (leader) tc::mbar_arrive_expect_tx(&c.full[stage], bytes);
                        tc::tma_load_2d_pair(s + BM * BK, &tmA, bar, kb * BK, w0, pol_w);
                        load_tokens(s, tmB, bar, kb * BK, ti.row0 + rank * BM, rows, pol_x);
                        load_tokens(s + rows * BK, tmB, bar, kb * BK, a.M, BM - rows, pol_x);
                    }
                    __syncwarp();
                }
            }
            // drain: this CTA's copies have landed (the even CTA's full barrier saw
            // every byte of both CTAs when its last phase completed)
            const int zero = 0;
            for (uint32_t i = it < STAGES ? 0 : it - STAGES; i < it; ++i) {
                const uint32_t stage = i % STAGES;
                if (!tc::mbar_wait(leader ? &c.full[stage] : &c.empty[stage], (i / STAGES) & 1u,
                                   &zero))
                    atomicExch(a.status, MOE_ERR_TIMEOUT);
            }
        } else if (warp == 1 || warp == 3) {
            if (leader) {
                // ---------------- MMA issuers (even CTA): 256 tokens x 128 weight rows,
                // warp 1 the first half of the columns, warp 3 the second
                const uint32_t half = warp >> 1;
                const uint32_t idesc = tc::idesc_e4m3_f32(NM, COLS / 2);
                uint32_t blk = 0;
                bool ok = true;
                for (int t = pair; t < total && ok; t += n_pairs) {
                    for (int kb = 0; kb < KB; ++kb, ++blk) {
                        const uint32_t as = blk & 1u, stage = blk % STAGES;
                        if (!tc::mbar_wait_warp(&c.acc_empty[as][half], ((blk >> 1) & 1u) ^ 1u,
                                                abort_flag) ||
                            !tc::mbar_wait_warp(&c.full[stage], (blk / STAGES) & 1u, abort_flag)) {
                            give_up(c, a.status);
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t x = tc::smem_u32(smem + stage * STAGE_BYTES);
                        const uint32_t w = x + BM * BK + half * (BM / 2) * BK;
                        if (tc::elect_one()) {
#pragma unroll
                            for (int k = 0; k < BK / 32; ++k)
                                tc::mma_e4m3_pair(tmem_base + as * COLS + half * (COLS / 2),
                                                  tc::desc_sw128(x + k * 32),
                                                  tc::desc_sw128(w + k * 32), idesc, k > 0);
                            tc::mma_commit_pair(&c.acc_full[as][half], 0x3);
                            tc::mma_commit_pair(&c.empty[stage], 0x3);
                        }
                        __syncwarp();
                    }
                }
                if (tc::elect_one()) tc::mma_commit_pair(&c.drain[half], 0x1);
                __syncwarp();
                const int zero = 0;
                if (!tc::mbar_wait(&c.drain[half], 0, &zero)) atomicExch(a.status, MOE_ERR_TIMEOUT);
            }
        } else if (warp == SCALE_WARP) {
            // ---------------- factors: per block sx[token] * sw of each half of the
            // columns, 4 tokens a lane, FB blocks a slot; the ring runs ahead of the
            // promotion, over tile borders too
            const int nb_n = (a.N + 127) / 128;
            const int sw_rows = GATE_UP ? 2 * nb_n : nb_n;
            uint32_t batch = 0;
            bool ok = true;
            for (int t = pair, i_t = 0; t < total && ok; t += n_pairs, ++i_t) {
                const Tile ti = listed_tile<NM>(c.list, c.tab, a.G, i_t, t);
                const float* sxp = a.sx + (size_t)(ti.row0 + rank * BM + lane) * KB;
                const int left = ti.len - rank * BM - lane;
                const int nb0 = GATE_UP ? ti.m : ti.m * 2;
                const int nb1 = GATE_UP ? nb_n + ti.m : min(ti.m * 2 + 1, nb_n - 1);
                const float* sw0 = a.sw + ((size_t)ti.g * sw_rows + nb0) * KB;
                const float* sw1 = a.sw + ((size_t)ti.g * sw_rows + nb1) * KB;
                for (int k0 = 0; k0 < KB; k0 += FB, ++batch) {
                    float x[4][FB], w0[FB], w1[FB];
#pragma unroll
                    for (int u = 0; u < FB; ++u) {
                        const bool in = k0 + u < KB;
                        w0[u] = in ? sw0[k0 + u] : 0.f;
                        w1[u] = in ? sw1[k0 + u] : 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i][u] = in && 32 * i < left ? sxp[(size_t)(32 * i) * KB + k0 + u]
                                                          : 0.f;
                    }
                    const uint32_t slot = batch % SLOTS;
                    ok = tc::mbar_wait_hot(&c.sc_empty[slot], ((batch / SLOTS) & 1u) ^ 1u,
                                           abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) {
                        give_up(c, a.status);
                        break;
                    }
#pragma unroll
                    for (int u = 0; u < FB; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            c.factor[slot][u][0][lane + 32 * i] = x[i][u] * w0[u];
                            c.factor[slot][u][1][lane + 32 * i] = x[i][u] * w1[u];
                        }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&c.sc_full[slot]);
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

template <bool GATE_UP, bool OUT_F32>
cudaError_t launch(const CUtensorMap& ma, const TokenMaps& mb, const Args& a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    auto kernel = block_many_kernel<GATE_UP, OUT_F32>;
    const cudaError_t err = allow_smem((const void*)kernel, SMEM, done, REGS);
    return err != cudaSuccess ? err : launch_pairs(kernel, sm_pairs(), THREADS, SMEM, s, ma, mb, a);
}

}  // namespace

cudaError_t launch_many(const BlockGemm& p, bool gate_up, cudaStream_t s) {
    const int w_rows = gate_up ? 2 * p.N : p.N;
    const int per_tile = gate_up ? BM : COLS;
    const Args a = {p.sx, p.sw, p.offsets, p.G, p.M, p.N, p.K, (p.N + per_tile - 1) / per_tile,
                    w_rows, p.out, p.out_scales, p.status, nullptr, 0};
    CUtensorMap ma;
    TokenMaps mb;
    if (!make_byte_map(&ma, p.wq, (uint64_t)p.G * w_rows, p.K, BM) ||
        !make_token_byte_maps(&mb, p.xq, p.M, p.K, 4))
        return cudaErrorInvalidValue;
    if (gate_up)
        return launch<true, false>(ma, mb, a, s);
    if (p.out_type == MOE_OUT_F32)
        return launch<false, true>(ma, mb, a, s);
    return launch<false, false>(ma, mb, a, s);
}

}  // namespace block
}  // namespace moe
