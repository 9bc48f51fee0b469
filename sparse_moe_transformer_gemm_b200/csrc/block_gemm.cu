// block_gemm.cu -- FP8 (e4m3) matrix products with an fp32 scale per block of
// 128, dense or grouped by row offsets, and the SwiGLU gate_up form whose
// result is quantised again, on pairs of SMs (tcgen05 cta_group::2).
//
//   out[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{c in block b} xq[m, c] wq[n, c]
//   gate_up:  h = SiLU(g) u in fp32, hq / sh its quantisation per 128 features
//
// The scales change with every block of 128 columns, so the tensor core sums one
// block at a time: four K = 32 MMAs of kind::f8f6f4 into a TMEM accumulator that
// starts from zero, which the promotion warps then read, multiply by
// sx[m, b] sw[n/128, b] and add to fp32 registers while the MMAs of the next
// block fill the other half of TMEM. The weight rows are the MMA's M (a thread
// of the promotion owns one weight row) and the tokens its N: a CTA's 128 weight
// rows lie in one block of rows, so the factor of a token's column is the same
// for the whole CTA, and a few tokens take a small N instead of a padded M.
//
// A pair tile takes 256 weight rows (128 a CTA) per accumulator:
//   WIDE  two accumulators against the same tokens, at most 128: gate_up's gate
//         and up rows (SiLU(g) u is then formed in registers), or two 256-row
//         tiles of a plain product;
//   TALL  one accumulator against at most 256 tokens: the same 256 columns of
//         TMEM per block and the same 128 accumulator registers a thread, with
//         32 instead of 40 KB through shared memory per block at a full tile.
//
// Per CTA (384 threads): warp 0 TMA producer, warp 1 TMEM owner (+ MMA issuer in
// the even CTA), warp 2 the scales: it forms the products of a block's two scales
// for every token in a ring in shared memory; warps 4-11 promotion and epilogue
// in two groups of four (one warp per TMEM lane quarter), each taking half of the
// tokens. The promotion's threads hold 128 accumulators, so the first four warps
// hand registers over (setmaxnreg). All waits are bounded.
#include <cudaTypedefs.h>

#include "internal.h"
#include "quant.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                // weight rows per CTA and accumulator
constexpr int BK = 128;                // columns per block = bytes per staged row
constexpr int A_BYTES = BM * BK;
constexpr int NBOX = 16;               // token rows of the smallest TMA box
constexpr int GROUPS = 2;              // promotion groups (4 warps each)
constexpr int SCALE_WARP = 2;
constexpr int PROMO_WARP = 4;          // the first one
constexpr int THREADS = 32 * (PROMO_WARP + 4 * GROUPS);
// registers a thread: 168 at launch; 3 * 168 = 72 + 2 * 216
constexpr int REGS_FEW = 72, REGS_MANY = 216;
static_assert(REGS_FEW + GROUPS * REGS_MANY == (1 + GROUPS) * 168, "no more than the launch gave");
constexpr int COLS = 256;              // TMEM columns per block
constexpr int CH = 16;                 // columns per promotion chunk
constexpr int NCH = COLS / GROUPS / CH;  // chunks per thread
constexpr int SLOTS = 4;               // scale ring
constexpr int EPI_BYTES = GROUPS * 2 * CH * BM * 2;  // two [16 tokens][128 rows] bf16 a group
constexpr int MAX_G = 257;             // 256 experts and a shared one
constexpr int MAX_STAGES = 6;

template <bool WIDE>
struct Shape {
    static constexpr int NM = WIDE ? 128 : 256;  // tokens per pair tile at most
    static constexpr int A_TILES = WIDE ? 2 : 1;
    static constexpr int STAGE_BYTES = A_TILES * A_BYTES + NM / 2 * BK;  // 40 / 32 KB
    static constexpr int STAGES = WIDE ? 5 : 6;
};

struct TokenMaps {
    CUtensorMap m[4];  // boxes of 16, 32, 64 and 128 rows
};

struct Ctrl {
    uint64_t full[MAX_STAGES];   // even CTA: TMA bytes of both CTAs landed
    uint64_t empty[MAX_STAGES];  // both CTAs: the pair MMAs finished reading the stage
    uint64_t acc_full[2];        // both CTAs: a block's sums are in TMEM
    uint64_t acc_empty[2];       // even CTA: every promotion warp of both CTAs has read them
    uint64_t sc_full[SLOTS];
    uint64_t sc_empty[SLOTS];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int total;
    int off[MAX_G + 1];
    int tile_start[MAX_G + 1];
    alignas(16) float scales[SLOTS][COLS];
    alignas(16) float4 hscale[GROUPS][64];  // gate_up: BlockScale of a token
};

template <bool WIDE>
constexpr int smem_bytes() {
    return Shape<WIDE>::STAGES * Shape<WIDE>::STAGE_BYTES + EPI_BYTES + 1024 + (int)sizeof(Ctrl);
}
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "fits in 227 KB");

struct Args {
    const float* sx;
    const float* sw;
    const int* offsets;
    int G, M, N, K;    // N: output features (gate_up: d_ff)
    int m_tiles;       // weight tiles of a group
    int w_rows;        // weight rows of a group
    void* out;
    float* out_scales;
    int* status;
};

struct Tile {
    int g, m, row0, len, n;  // n: MMA N, a multiple of 32
};

// Tile t: token tiles fastest (tiles that read the same weights are neighbours in
// time, so HBM gives them once and L2 the other times), then weight tiles, then
// groups. A group's rows split into nt = ceil(rows / NM) token tiles, all but
// the last a multiple of 32 rows and as equal as that allows.
template <int NM>
__device__ __forceinline__ Tile tile_of(const Ctrl& c, int G, int t) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c.tile_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int rows = c.off[lo + 1] - c.off[lo];
    const int nt = (rows + NM - 1) / NM;
    const int units = (rows + 31) / 32;
    int q = (units + nt - 1) / nt;
    if (32 * q * (nt - 1) >= rows) q = NM / 32;
    const int local = t - c.tile_start[lo];
    const int j = local % nt;
    Tile r;
    r.g = lo;
    r.m = local / nt;
    r.row0 = c.off[lo] + j * 32 * q;
    r.len = j < nt - 1 ? 32 * q : rows - 32 * q * (nt - 1);
    r.n = (r.len + 31) & ~31;
    return r;
}

__device__ __forceinline__ void give_up(Ctrl& c, int* status) {
    *reinterpret_cast<volatile int*>(&c.abort) = 1;
    atomicExch(status, MOE_ERR_TIMEOUT);
}

// acc += d * s, two columns at a time (d: TMEM words, s: shared memory).
__device__ __forceinline__ void promote16(uint64_t (&acc)[CH / 2], const uint32_t (&d)[CH],
                                          const float* s) {
#pragma unroll
    for (int i = 0; i < CH / 4; ++i) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s + 4 * i);
        uint64_t a, b;
        asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "r"(d[4 * i]), "r"(d[4 * i + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "r"(d[4 * i + 2]), "r"(d[4 * i + 3]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[2 * i]) : "l"(a), "l"((uint64_t)f.x));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[2 * i + 1]) : "l"(b), "l"((uint64_t)f.y));
    }
}
__device__ __forceinline__ float lane_of(const uint64_t (&acc)[CH / 2], int i) {
    return __uint_as_float((uint32_t)(acc[i >> 1] >> (32 * (i & 1))));
}

// tmA: weights [G * w_rows, K] bytes, box 128 x 128; tmB: tokens [M, K] bytes.
template <bool GATE_UP, bool WIDE, bool OUT_F32>
__global__ void __launch_bounds__(THREADS, 1)
block_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ TokenMaps tmB,
                  const Args a) {
    static_assert(WIDE || !GATE_UP, "gate_up pairs its two accumulators");
    using S = Shape<WIDE>;
    pdl_launch_and_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* epi = smem + S::STAGES * S::STAGE_BYTES;
    Ctrl& c = *reinterpret_cast<Ctrl*>(epi + EPI_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(tc::cluster_ctarank() & 1u);
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    const int KB = (a.K + BK - 1) / BK;

    // ---- prologue: tile table (warp 0), barriers and TMEM (warp 1), in both CTAs
    if (warp == 0) {
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
                if (g < a.G) cnt = max(0, (offset(g + 1) - o + S::NM - 1) / S::NM) * a.m_tiles;
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
            c.abort = 0;
            tc::prefetch_tensormap(&tmA);
            for (int m = 0; m < 4; ++m) tc::prefetch_tensormap(&tmB.m[m]);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < S::STAGES; ++s) {
                tc::mbar_init(&c.full[s], 1);
                tc::mbar_init(&c.empty[s], 1);
            }
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(&c.acc_full[i], 1);
                tc::mbar_init(&c.acc_empty[i], 2 * 4 * GROUPS);
            }
            for (int i = 0; i < SLOTS; ++i) {
                tc::mbar_init(&c.sc_full[i], 1);
                tc::mbar_init(&c.sc_empty[i], 4 * GROUPS);
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
    const uint32_t tmem_base = c.tmem_base;
    const int total = c.total;
    const volatile int* abort_flag = &c.abort;
    // first weight row of a tile's accumulator p, within its group, for this CTA
    auto first_row = [&](int m, int p) {
        if (GATE_UP) return p * a.N + m * 2 * BM + rank * BM;
        return m * S::A_TILES * 2 * BM + p * 2 * BM + rank * BM;
    };
    // whether the pair's accumulator 1 has rows (always in gate_up)
    auto two = [&](int m) { return GATE_UP || (WIDE && m * 4 * BM + 2 * BM < a.N); };

    if (warp >= PROMO_WARP) {
        tc::regs_inc<REGS_MANY>();
        // ---------------- promotion and epilogue: lane = one weight row. Group grp
        // takes the tokens [grp * n/2, (grp + 1) * n/2) in chunks of 16; chunk i of
        // accumulator p is acc[p * NCH / 2 + i] (WIDE) or acc[i] (TALL).
        const int quad = warp & 3, grp = (warp - PROMO_WARP) >> 2;
        const int et = threadIdx.x - 32 * PROMO_WARP - 128 * grp;  // 0..127 within the group
        const int bar = 1 + grp;
        const int row = quad * 32 + lane;             // weight row within the CTA's 128
        const uint32_t lane_base = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint32_t acc_empty0 = tc::map_to_cta(tc::smem_u32(&c.acc_empty[0]), 0);
        uint32_t blk = 0;
        for (int t = pair; t < total; t += n_pairs) {
            const Tile ti = tile_of<S::NM>(c, a.G, t);
            const int half = ti.n / 2, col0 = grp * half;
            const int chunks = half / CH;
            const bool second = WIDE && two(ti.m);
            auto live = [&](int i) {
                return WIDE ? (i < NCH / 2 ? i < chunks : second && i - NCH / 2 < chunks)
                            : i < chunks;
            };
            auto column = [&](int i) {
                return WIDE ? (i < NCH / 2 ? col0 + i * CH : COLS / 2 + col0 + (i - NCH / 2) * CH)
                            : col0 + i * CH;
            };
            uint64_t acc[NCH][CH / 2];
#pragma unroll
            for (int i = 0; i < NCH; ++i)
#pragma unroll
                for (int j = 0; j < CH / 2; ++j) acc[i][j] = 0;
            bool ok = true;
            for (int kb = 0; kb < KB; ++kb, ++blk) {
                const uint32_t as = blk & 1u, slot = blk % SLOTS;
                ok = tc::mbar_wait_hot(&c.sc_full[slot], (blk / SLOTS) & 1u, abort_flag) &&
                     tc::mbar_wait_hot(&c.acc_full[as], (blk >> 1) & 1u, abort_flag);
                ok = __all_sync(0xffffffffu, ok);  // the warp stays together
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t tb = lane_base + as * COLS;
                const float* sc = c.scales[slot];
#pragma unroll
                for (int i = 0; i < NCH; i += 2) {
                    if (!live(i)) continue;
                    uint32_t d0[CH], d1[CH];
                    tc::tmem_ld16(tb + column(i), d0);
                    if (live(i + 1)) tc::tmem_ld16(tb + column(i + 1), d1);
                    tc::tmem_ld_wait();
                    promote16(acc[i], d0, sc + column(i));
                    if (live(i + 1)) promote16(acc[i + 1], d1, sc + column(i + 1));
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive_cluster_read(acc_empty0 + as * 8);
                    tc::mbar_arrive(&c.sc_empty[slot]);
                }
            }
            // a warp that gave up takes its group with it
            if (tc::bar_any(bar, 128, !ok)) {
                give_up(c, a.status);
                break;
            }
            const int rows_left = ti.len - col0;  // valid tokens of this group's half
            const long tok0 = ti.row0 + col0;
            if constexpr (GATE_UP) {
                const int f0 = ti.m * 2 * BM + rank * BM;  // first feature of the CTA's block
                float4* hs = c.hscale[grp];
                uint8_t* tile = epi + grp * (EPI_BYTES / GROUPS);  // [64 tokens][128 features]
                // before that: a token's largest |h| of each lane quarter
                uint32_t (*amax)[4] = reinterpret_cast<uint32_t(*)[4]>(tile);
#pragma unroll
                for (int i = 0; i < NCH / 2; ++i) {
                    if (i >= chunks) continue;
                    uint32_t mx = 0;
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        const float h0 = silu_mul(lane_of(acc[i], j), lane_of(acc[i + NCH / 2], j));
                        const float h1 =
                            silu_mul(lane_of(acc[i], j + 1), lane_of(acc[i + NCH / 2], j + 1));
                        acc[i][j / 2] = ((uint64_t)f32_bits(h1) << 32) | f32_bits(h0);
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
                if (et < half) {
                    const uint4 m = *reinterpret_cast<const uint4*>(amax[et]);
                    const BlockScale b =
                        block_scale(f32_from_bits(max(max(m.x, m.y), max(m.z, m.w))));
                    hs[et] = make_float4(b.a, b.inv, b.move, b.scale);
                    if (et < rows_left && f0 < a.N)
                        a.out_scales[(tok0 + et) * (a.N / 128) + (f0 >> 7)] = b.scale;
                }
                tc::bar_sync(bar, 128);
#pragma unroll
                for (int i = 0; i < NCH / 2; ++i) {
                    if (i >= chunks) continue;
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const float4 v = hs[i * CH + j];
                        const BlockScale b = {v.w, v.x, v.y, v.z};
                        tile[(i * CH + j) * BM + row] =
                            (uint8_t)e4m3x2_of(block_quotient(b, lane_of(acc[i], j)), 0.f);
                    }
                }
                tc::bar_sync(bar, 128);
                if (f0 < a.N)
                    for (int id = et; id < half * (BM / 16); id += 128) {
                        const int n = id / (BM / 16), ch = id % (BM / 16);
                        if (n < rows_left)
                            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) +
                                                      (tok0 + n) * a.N + f0 + ch * 16) =
                                *reinterpret_cast<const uint4*>(tile + n * BM + ch * 16);
                    }
                // (the next tile's bar_any comes before the next writes here)
            } else {
                const bool vec = !OUT_F32 && a.N % 8 == 0;
                uint16_t* tile = reinterpret_cast<uint16_t*>(epi + grp * (EPI_BYTES / GROUPS));
                int buf = 0;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    if (!live(i)) continue;
                    const int p = WIDE && i >= NCH / 2 ? 1 : 0;
                    const int n0 = first_row(ti.m, p);      // first output column
                    const int t0 = (i - p * (NCH / 2)) * CH;  // first token of the chunk
                    if (vec) {
                        // through a [16 tokens][128 rows] tile to 16-byte stores;
                        // two tiles, so one barrier per chunk
                        uint16_t* o = tile + buf * (CH * BM);
#pragma unroll
                        for (int j = 0; j < CH; ++j)
                            o[j * BM + row] = float_to_bf16_bits(lane_of(acc[i], j));
                        tc::bar_sync(bar, 128);
#pragma unroll
                        for (int q = 0; q < CH * BM / 8 / 128; ++q) {
                            const int id = et + 128 * q;
                            const int n = id / (BM / 8), ch = id % (BM / 8);
                            if (t0 + n < rows_left && n0 + ch * 8 < a.N)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                          (tok0 + t0 + n) * a.N + n0 + ch * 8) =
                                    *reinterpret_cast<const uint4*>(o + n * BM + ch * 8);
                        }
                        buf ^= 1;
                    } else if (n0 + row < a.N) {
#pragma unroll
                        for (int j = 0; j < CH; ++j)
                            if (t0 + j < rows_left) {
                                const long at = (tok0 + t0 + j) * a.N + n0 + row;
                                if (OUT_F32)
                                    static_cast<float*>(a.out)[at] = lane_of(acc[i], j);
                                else
                                    static_cast<uint16_t*>(a.out)[at] =
                                        float_to_bf16_bits(lane_of(acc[i], j));
                            }
                    }
                }
            }
        }
    } else {
        tc::regs_dec<REGS_FEW>();
        if (warp == 0) {
            if (lane == 0) {
                // ---------------- producer: this CTA's weight rows and token half
                const uint64_t pol_w = tc::policy_evict_first();
                const uint64_t pol_x = tc::policy_evict_last();
                int stage = 0;
                uint32_t phase = 0;
                uint32_t parity[S::STAGES] = {};
                bool issued[S::STAGES] = {};
                bool ok = true;
                for (int t = pair; t < total && ok; t += n_pairs) {
                    const Tile ti = tile_of<S::NM>(c, a.G, t);
                    const int half = ti.n / 2;
                    const int tiles = WIDE && two(ti.m) ? 2 : 1;
                    const int w0 = ti.g * a.w_rows + first_row(ti.m, 0);
                    const int w1 = ti.g * a.w_rows + first_row(ti.m, 1);
                    const uint32_t bytes = 2u * (tiles * A_BYTES + half * BK);
                    for (int kb = 0; kb < KB; ++kb) {
                        if (!tc::mbar_wait_hot(&c.empty[stage], phase ^ 1u, abort_flag)) {
                            give_up(c, a.status);
                            ok = false;
                            break;
                        }
                        const uint32_t bar = tc::map_to_cta(tc::smem_u32(&c.full[stage]), 0);
                        uint8_t* s = smem + stage * S::STAGE_BYTES;
                        uint8_t* sb = s + S::A_TILES * A_BYTES;
                        if (leader) tc::mbar_arrive_expect_tx(&c.full[stage], bytes);
                        tc::tma_load_2d_pair(s, &tmA, bar, kb * BK, w0, pol_w);
                        if (tiles == 2) tc::tma_load_2d_pair(s + A_BYTES, &tmA, bar, kb * BK, w1, pol_w);
                        for (int o = 0; o < half;) {
                            const int rem = half - o;
                            const int lg = rem >= 128 ? 3 : rem >= 64 ? 2 : rem >= 32 ? 1 : 0;
                            tc::tma_load_2d_pair(sb + o * BK, &tmB.m[lg], bar, kb * BK,
                                                 ti.row0 + rank * half + o, pol_x);
                            o += NBOX << lg;
                        }
                        issued[stage] = true;
                        parity[stage] = phase;
                        if (++stage == S::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                // drain: this CTA's copies have landed (the even CTA's full barrier saw
                // every byte of both CTAs when its last phase completed)
                const int zero = 0;
                for (int s = 0; s < S::STAGES; ++s)
                    if (issued[s] && !tc::mbar_wait(leader ? &c.full[s] : &c.empty[s], parity[s], &zero))
                        atomicExch(a.status, MOE_ERR_TIMEOUT);
            }
        } else if (warp == 1) {
            if (lane == 0 && leader) {
                // ---------------- MMA issuer (even CTA), M = 256 across the pair
                int stage = 0;
                uint32_t phase = 0, blk = 0;
                bool ok = true;
                for (int t = pair; t < total && ok; t += n_pairs) {
                    const Tile ti = tile_of<S::NM>(c, a.G, t);
                    const uint32_t idesc = tc::idesc_e4m3_f32(2 * BM, ti.n);
                    const bool second = WIDE && two(ti.m);
                    for (int kb = 0; kb < KB; ++kb, ++blk) {
                        const uint32_t as = blk & 1u;
                        if (!tc::mbar_wait_hot(&c.acc_empty[as], ((blk >> 1) & 1u) ^ 1u, abort_flag) ||
                            !tc::mbar_wait_hot(&c.full[stage], phase, abort_flag)) {
                            give_up(c, a.status);
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t d = tmem_base + as * COLS;
                        const uint32_t a_addr = tc::smem_u32(smem + stage * S::STAGE_BYTES);
                        const uint32_t b_addr = a_addr + S::A_TILES * A_BYTES;
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k) {
                            const uint64_t bd = tc::desc_sw128(b_addr + k * 32);
                            tc::mma_e4m3_pair(d, tc::desc_sw128(a_addr + k * 32), bd, idesc, k > 0);
                            if (second)
                                tc::mma_e4m3_pair(d + COLS / 2,
                                                  tc::desc_sw128(a_addr + A_BYTES + k * 32), bd, idesc,
                                                  k > 0);
                        }
                        tc::mma_commit_pair(&c.empty[stage], 0x3);
                        tc::mma_commit_pair(&c.acc_full[as], 0x3);
                        if (++stage == S::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                tc::mma_commit_pair(&c.drain, 0x1);
                const int zero = 0;
                if (!tc::mbar_wait(&c.drain, 0, &zero)) atomicExch(a.status, MOE_ERR_TIMEOUT);
            }
        } else if (warp == SCALE_WARP) {
            // ---------------- scales: per block the products sx[token] * sw of this
            // CTA's weight rows, U blocks loaded at a time. The ring runs ahead of
            // the promotion, over tile borders too.
            constexpr int TPL = S::NM / 32;    // tokens per lane
            constexpr int U = WIDE ? 4 : 2;    // blocks loaded at a time
            const int nb_n = (a.N + 127) / 128;
            const int sw_rows = GATE_UP ? 2 * nb_n : nb_n;
            uint32_t blk = 0;
            bool ok = true;
            for (int t = pair; t < total && ok; t += n_pairs) {
                const Tile ti = tile_of<S::NM>(c, a.G, t);
                const float* swp[S::A_TILES];
#pragma unroll
                for (int p = 0; p < S::A_TILES; ++p) {
                    const int nb = min(first_row(ti.m, p) / BM, sw_rows - 1);
                    swp[p] = a.sw + ((size_t)ti.g * sw_rows + nb) * KB;
                }
                for (int k0 = 0; k0 < KB && ok; k0 += U) {
                    float x[TPL][U], w[S::A_TILES][U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
#pragma unroll
                        for (int p = 0; p < S::A_TILES; ++p)
                            w[p][u] = k0 + u < KB ? swp[p][k0 + u] : 0.f;
#pragma unroll
                        for (int i = 0; i < TPL; ++i) {
                            const int n = lane + 32 * i;
                            x[i][u] = k0 + u < KB && n < ti.len
                                          ? a.sx[(size_t)(ti.row0 + n) * KB + k0 + u] : 0.f;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (k0 + u >= KB || !ok) continue;
                        const uint32_t slot = blk % SLOTS;
                        ok = tc::mbar_wait_hot(&c.sc_empty[slot], ((blk / SLOTS) & 1u) ^ 1u, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) {
                            give_up(c, a.status);
                            continue;
                        }
#pragma unroll
                        for (int i = 0; i < TPL; ++i)
#pragma unroll
                            for (int p = 0; p < S::A_TILES; ++p)
                                c.scales[slot][p * (COLS / 2) + lane + 32 * i] = x[i][u] * w[p][u];
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

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

// Row-major [rows, cols] bytes, box of box_rows rows x 128 bytes, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols};
    cuuint32_t box[2] = {(cuuint32_t)BK, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_pairs() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return (n > 1 ? n : 148) / 2;
}

template <bool GATE_UP, bool WIDE, bool OUT_F32>
cudaError_t launch(const BlockGemm& p, cudaStream_t s) {
    const int w_rows = GATE_UP ? 2 * p.N : p.N;
    const int per_tile = GATE_UP ? 2 * BM : Shape<WIDE>::A_TILES * 2 * BM;
    const Args a = {p.sx, p.sw, p.offsets, p.G, p.M, p.N, p.K, (p.N + per_tile - 1) / per_tile,
                    w_rows, p.out, p.out_scales, p.status};
    CUtensorMap ma;
    TokenMaps mb;
    if (!make_map(&ma, p.wq, (uint64_t)p.G * w_rows, p.K, BM)) return cudaErrorInvalidValue;
    for (int lg = 0; lg < 4; ++lg)
        if (!make_map(&mb.m[lg], p.xq, p.M, p.K, NBOX << lg)) return cudaErrorInvalidValue;
    const int smem = smem_bytes<WIDE>();
    auto kernel = block_gemm_kernel<GATE_UP, WIDE, OUT_F32>;
    cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * sm_pairs(), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
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
    err = cudaLaunchKernelEx(&cfg, kernel, ma, mb, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_gemm(const BlockGemm& p, cudaStream_t s) {
    // more than 128 rows a group on average: token tiles of up to 256
    if ((long)p.M > 128L * p.G)
        return p.out_type == MOE_OUT_F32 ? launch<false, false, true>(p, s)
                                         : launch<false, false, false>(p, s);
    return p.out_type == MOE_OUT_F32 ? launch<false, true, true>(p, s)
                                     : launch<false, true, false>(p, s);
}
cudaError_t launch_block_gate_up(const BlockGemm& p, cudaStream_t s) {
    return launch<true, true, false>(p, s);
}

}  // namespace moe
