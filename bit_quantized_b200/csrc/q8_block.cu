// Block-scaled FP8 (e4m3 codes, one scale per 128 values of a token and per
// 128 x 128 block of a weight): quantizers, the dense linear and the linear
// grouped by expert.
//
//   act     Sx[j, t] = max(fl32(absmax of x[t, 128 j ..] / 448), 1e-8)
//   weight  Sw[i, j] = the same over rows 128 i .. and columns 128 j ..
//   linear  y[t, n] = sum_j Sx[j, t] Sw[n / 128, j] p_j,
//           p_j = sum over the 128 k of group j of qx[t, k] qw[n, k]
//
// The scales change along K, so a GEMM cannot leave them to its epilogue:
// each p_j is one tcgen05 accumulation of 128 values in TMEM, and CUDA cores
// add it, scaled, to fp32 sums in registers (a "promotion").  TMEM holds two
// p_j, so the tensor cores work on group j + 1 while group j is promoted.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "q8_block.cuh"
#include "q8_internal.h"
#include "q8_tile.cuh"

namespace q8 {
namespace {

constexpr int kBM = 128;    // MMA M per CTA (TMEM lanes)
constexpr int kBKB = 128;   // bytes of K per stage: one scale group, one swizzle row

// ============================================================================
// Quantizers
// ============================================================================
//
// Both read each value once and hold it in registers between the absmax and
// the codes.  16 lanes share a group of 128 values (16 bytes of a 16-bit type
// each).

// Bytes in flight bound them: CTAs of 32 KB of input, four or five per SM
// (4096x8192 bf16 activations: 21.4 us with 16 KB, 19.1 with 32 = 5.3 TB/s, 22.9
// with 64; 8192x8192 bf16 weights: 38.3 us = 5.3 TB/s, with 64 KB 43.0; persistent
// forms that load a tile ahead: 22.9 and 47.2; fp32: 6.1 and 6.3 TB/s).
constexpr int kActRows = 32;   // rows per block: the scales of a group leave as one run

// Activation: 32 rows x 256 H columns per block; a warp takes four rows, H times
// 512 bytes of each (H = 2 for 16-bit inputs: 32 KB per block).  The 4 H maxima
// of a lane are reduced together: lanes 8, 4 (and 2) apart split them, so that
// each lane ends with one row's and computes that group's scale alone; the
// scales go round by shuffles.  The scales are group-major, so they are
// gathered in shared memory and written as runs of 32 rows.
template <typename T, int H>
__global__ void __launch_bounds__(256)
act_block_quant_kernel(const T* X, int64_t m, int64_t k, int64_t ldx, uint8_t* __restrict__ codes,
                       float* __restrict__ scale) {
    constexpr int N = 4 * H;                 // pieces: row i / H, columns i % H
    __shared__ float s_sh[2 * H][kActRows];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kActRows + warp * 4;
    const int64_t col0 = static_cast<int64_t>(blockIdx.y) * (256 * H) + lane * 8;
    pdl_wait();
    pdl_launch_dependents();
    Eight<T> v[N];
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t r = row0 + i / H, col = col0 + i % H * 256;
        if (r < m && col < k) v[i].load(X + r * ldx + col);
        else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = v[i].absmax();
    int left = N, mine_i = 0;                // this lane's piece
#pragma unroll
    for (int o = 8; o; o >>= 1) {
        if (left > 1) {
            const bool up = lane & o;
            left /= 2;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < left) a[i] = fmaxf(up ? a[i + left] : a[i], __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + left], o));
            if (up) mine_i += left;
        } else {
            a[0] = fmaxf(a[0], __shfl_xor_sync(0xffffffffu, a[0], o));
        }
    }
    const BlockScale mine = block_scale(a[0]);
    if (lane % (16 / N) == 0) s_sh[mine_i % H * 2 + lane / 16][warp * 4 + mine_i / H] = mine.S;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int from = (lane & 16) + i * (16 / N);
        BlockScale s;
        s.S = __shfl_sync(0xffffffffu, mine.S, from);
        s.R = __shfl_sync(0xffffffffu, mine.R, from);
        s.Rlo = __shfl_sync(0xffffffffu, mine.Rlo, from);
        float f[8];
        v[i].values(f);
        const uint2 w = make_uint2(block_codes4(f[0], f[1], f[2], f[3], s), block_codes4(f[4], f[5], f[6], f[7], s));
        const int64_t r = row0 + i / H, col = col0 + i % H * 256;
        if (r < m && col < k) *reinterpret_cast<uint2*>(codes + r * k + col) = w;
    }
    __syncthreads();
    if (threadIdx.x < 2 * H * kActRows) {
        const int g = threadIdx.x / kActRows, i = threadIdx.x % kActRows;
        const int64_t j = static_cast<int64_t>(blockIdx.y) * 2 * H + g, r = static_cast<int64_t>(blockIdx.x) * kActRows + i;
        if (j * kBlock < k && r < m) scale[j * m + r] = s_sh[g][i];
    }
}

// Weight: one 128 x 128 block per CTA, eight passes of 16 rows.  blockIdx.z is
// the matrix of a stack; its row blocks start anew.
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2)
weight_block_quant_kernel(const T* __restrict__ W, int64_t n, int64_t k, int64_t ldw, uint8_t* __restrict__ codes,
                          float* __restrict__ scale, int64_t nb, int64_t kb) {
    __shared__ float m_sh[8];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t e = blockIdx.z, bi = blockIdx.y, bj = blockIdx.x;
    const int64_t col = bj * kBlock + (threadIdx.x % 16) * 8;
    const int64_t r0 = bi * kBlock + threadIdx.x / 16;
    Eight<T> v[8];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r < n && col < k) v[i].load(W + (e * n + r) * ldw + col);
        else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, v[i].absmax());
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane == 0) m_sh[warp] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) a = fmaxf(a, m_sh[w]);
    const BlockScale s = block_scale(a);
    if (threadIdx.x == 0) scale[(e * nb + bi) * kb + bj] = s.S;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r < n && col < k) {
            float f[8];
            v[i].values(f);
            *reinterpret_cast<uint2*>(codes + (e * n + r) * k + col) =
                make_uint2(block_codes4(f[0], f[1], f[2], f[3], s), block_codes4(f[4], f[5], f[6], f[7], s));
        }
    }
}

// ============================================================================
// Tile kernel: 128 x BN output tiles, persistent
// ============================================================================
//
// Roles as in the rowwise tile GEMM (TMA producer, MMA issuer), but eight
// promotion warps: a warp reads its 32-lane quarter of TMEM (its threads' token
// rows) and half of the tile's columns, BN / 2 fp32 sums per thread.  Every K
// group is handed over through the accumulator barriers, and the sums leave
// through TMA stores when the tile is done.
//
// One CTA per tile, not a CTA pair: with two accumulators in TMEM the MMA of
// group j + 2 waits for the promotion of group j, and across a pair that round
// trip (commit to both CTAs, arrivals from both) takes about 1400 cycles per two
// groups of 512 each; inside one CTA it fits under the MMAs, which is worth
// more than the pair's smaller operand traffic.

constexpr int kPromoWarps = 8;
constexpr int kTileThreads = 128 + 32 * kPromoWarps;
// Registers: 384 threads launch with 168 each (64,512); the first warpgroup
// (TMA, two MMA warps, an idle one) keeps 72 and the two promotion warpgroups take 216
// (128 x 72 + 256 x 216 = 64,512), which holds 128 fp32 sums per thread.
constexpr int kTileRegsLow = 72, kTileRegsHigh = 216;

struct BlockParams {
    int m, n;
    const float* sx;      // [kb][m]
    const float* sw;      // [experts][nb][kb]
    const float* bias;    // [experts * n] or null
    __nv_bfloat16* y;
    int64_t ldy;
    int* status;
};

template <int BN>
struct BlockTileCfg {
    static constexpr int A_BYTES = kBM * kBKB;
    static constexpr int B_BYTES = BN * kBKB;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STORE = kPromoWarps * 2048;       // output staging: one 32 x 32 chunk per warp
    static constexpr int STAGES_RAW = (227 * 1024 - STORE - 1024 - 6 * 1024) / STAGE;
    static constexpr int STAGES = STAGES_RAW > 8 ? 8 : STAGES_RAW;
    static constexpr int TMEM_COLS = BN <= 128 ? 256 : 512;
    static constexpr int CW = BN / 2;                      // columns per promotion warp
    // Groups that the scales are fetched ahead of their use: a group of narrow
    // tiles is short, and wide ones leave few registers (512x4096x4096: 14.5 us
    // with four groups ahead, 14.0 with eight; 4096x8192x8192: 299 us with four,
    // which spill inside the group loop, 245 with two).
    static constexpr int AHEAD = BN == 128 ? 8 : BN == 192 ? 4 : 2;
    // 96 columns may reach into a second weight block (at a multiple of 32).
    static constexpr bool TWO = CW % 128 != 0 && 128 % CW != 0;
    static constexpr int SMEM = STAGES * STAGE + STORE + 1024;
    static_assert(BN == 128 || BN == 192 || BN == 256, "BN");
    static_assert(STAGES >= 2, "the two issuing warps share the stages' barriers");
};

template <int BN, bool GROUPED>
__global__ void __launch_bounds__(kTileThreads, 1)
gemm_block_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmY, int use_tmy, const BlockParams p, int num_kb,
                       int tiles_m, int tiles_n, const int32_t* group_offsets, int experts) {
    using C = BlockTileCfg<BN>;
    __shared__ int g_off[GROUPED ? kMaxGroupedExperts + 1 : 1];
    __shared__ int g_mt[GROUPED ? kMaxGroupedExperts + 1 : 1];
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    __shared__ __align__(8) uint64_t full_bar[C::STAGES];
    __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[2];
    __shared__ __align__(8) uint64_t tempty_bar[2];
    __shared__ __align__(8) uint64_t drain_bar[2];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = warp_index();
    const int lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], kPromoWarps);
        }
        mbar_init(&drain_bar[0], 1);
        mbar_init(&drain_bar[1], 1);
        abort_sh = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
        tmem_relinquish();
    }
    if constexpr (GROUPED) {
        // The routing offsets come from the previous kernels.
        pdl_wait();
        if (warp == 2) build_group_map(group_offsets, experts, p.m, kBM, g_off, g_mt);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;
    pdl_launch_dependents();

    const int num_tiles = GROUPED ? g_mt[GROUPED ? experts : 0] * tiles_n : tiles_m * tiles_n;
    const int first_tile = static_cast<int>(blockIdx.x), step = static_cast<int>(gridDim.x);
    auto tile_ref = [&](int tile) -> TileRef {
        if constexpr (GROUPED) return grouped_tile(tile, g_off, g_mt, experts, kBM, BN, p.n);
        else return dense_tile(tile, tiles_m, kBM, BN, p.m);
    };
    if (warp == 0) {
        reg_dealloc<kTileRegsLow>();
        // ------------------------------------------------ TMA producer
        if (elect_one()) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            // The weights do not depend on the previous kernel: the first ring
            // of the first tile's weight slices goes out before the wait.
            int npre = 0;
            if constexpr (!GROUPED) {
                if (first_tile < num_tiles) {
                    const TileRef tr0 = tile_ref(first_tile);
                    npre = num_kb < C::STAGES ? num_kb : C::STAGES;
                    for (int s = 0; s < npre; ++s) {
                        mbar_arrive_expect_tx(&full_bar[s], C::STAGE);
                        tma_load_2d(smem + s * C::STAGE + C::A_BYTES, &tmB, &full_bar[s], s * kBKB, tr0.b_row);
                    }
                }
            }
            pdl_wait();
            uint32_t issued = (1u << npre) - 1u, last_par = 0;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = first_tile; tile < num_tiles && ok; tile += step) {
                const TileRef tr = tile_ref(tile);
                for (int kb = 0; kb < num_kb; ++kb) {
                    const bool pre = tile == first_tile && kb < npre;   // weight slice already out
                    if (!pre && !mbar_wait_short(&empty_bar[stage], phase ^ 1, &abort_sh, p.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = smem + stage * C::STAGE;
                    if (!pre) mbar_arrive_expect_tx(&full_bar[stage], C::STAGE);
                    tma_load_2d(sa, &tmA, &full_bar[stage], kb * kBKB, tr.a_row);
                    if (!pre) tma_load_2d(sa + C::A_BYTES, &tmB, &full_bar[stage], kb * kBKB, tr.b_row);
                    issued |= 1u << stage;
                    last_par = (last_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok)   // the loads already issued land before the CTA leaves
                for (int s = 0; s < C::STAGES; ++s)
                    if (issued & (1u << s)) mbar_wait(&full_bar[s], (last_par >> s) & 1, nullptr, nullptr);
        }
        __syncwarp();
    } else if (warp < 3) {
        reg_dealloc<kTileRegsLow>();
        // ------------------------------------------------ MMA issuers
        // Two warps take the K groups in turn, each with an accumulator of its
        // own: an issuing warp spends about 200 cycles on every commit, which
        // would otherwise stand between a group's MMAs and the next one's
        // (512x4096x4096: 15.2 -> 13.2 us).  A stage's barrier is waited for by
        // either warp in turn, which its parity bears because the accumulator
        // comes first: it is free once the promotion of two groups ago is over,
        // and with it every earlier use of the stage.  The whole warp runs the loop and one lane issues: descriptors then stay in
        // uniform registers, without which an MMA takes about 75 cycles to issue.
        const int w = warp - 1;
        const bool leader = elect_one();
        const uint32_t idesc = make_idesc(1, 0, 0, kBM, BN);
        const uint32_t d = tmem_base + w * BN;
        int stage = 0, turn = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        for (int tile = first_tile; tile < num_tiles && ok; tile += step) {
            for (int kb = 0; kb < num_kb; ++kb) {
                if (turn == w) {
                    if (!__all_sync(0xffffffffu, mbar_wait_short(&tempty_bar[w], bphase ^ 1, &abort_sh, p.status) &&
                                                 mbar_wait_short(&full_bar[stage], phase, &abort_sh, p.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + stage * C::STAGE);
                    const uint64_t ad = sdesc_kmajor_sw128(sa);
                    const uint64_t bd = sdesc_kmajor_sw128(sa + C::A_BYTES);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < kBKB / 32; ++ks)
                            mma_issue<kKindF8>(d, ad + 2 * ks, bd + 2 * ks, idesc, ks != 0);
                        tc_commit(&tfull_bar[w]);
                        tc_commit(&empty_bar[stage]);
                    }
                    __syncwarp();
                    bphase ^= 1;
                }
                turn ^= 1;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && leader) {
            // Abort: wait for the MMAs already issued before TMEM is freed.
            tc_commit(&drain_bar[w]);
            mbar_wait(&drain_bar[w], 0, nullptr, nullptr);
        }
        __syncwarp();
    } else if (warp < 4) {
        reg_dealloc<kTileRegsLow>();
    } else {
        reg_alloc<kTileRegsHigh>();
        // ------------------------------------------------ promotion and epilogue
        pdl_wait();
        const int q = warp & 3, half = (warp - 4) >> 2;
        uint8_t* store = smem + C::STAGES * C::STAGE + (warp - 4) * 2048;
        const int nb_all = (p.n + kBlock - 1) / kBlock;
        int buf = 0;
        uint32_t bphase = 0;
        bool ok = true;
        for (int tile = first_tile; tile < num_tiles && ok; tile += step) {
            const TileRef tr = tile_ref(tile);
            const int row0 = tr.a_row + q * 32;
            const int row = row0 + lane;
            const int ncol = tr.n_tile + half * C::CW;         // this warp's first column
            int nb = ncol / kBlock;
            if (nb >= nb_all) nb = nb_all - 1;                 // columns past n: computed, not stored
            const int e = GROUPED ? tr.col_off / p.n : 0;
            const float* sx = p.sx + (row < p.m ? row : p.m - 1);
            const float* sw = p.sw + (static_cast<int64_t>(e) * nb_all + nb) * num_kb;
            const int64_t to_next = nb + 1 < nb_all ? num_kb : 0;   // the next block's scales
            const int cut = (ncol / kBlock + 1) * kBlock - ncol;    // columns before it
            float2 acc[C::CW / 2];
#pragma unroll
            for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            // Scales are fetched AHEAD groups before their use.  The loads are
            // volatile and the products are formed at the use: left to itself,
            // the compiler forms them right behind the loads, and every group
            // then waits for memory.
            float s_a[C::AHEAD], s_b[C::AHEAD], s_c[C::TWO ? C::AHEAD : 1];
            auto fetch = [&](int j) {
                s_a[j] = ld_act_scale(sx);
                s_b[j] = ld_weight_scale(sw);
                if constexpr (C::TWO) s_c[j] = ld_weight_scale(sw + to_next);
            };
#pragma unroll
            for (int j = 0; j < C::AHEAD; ++j) {
                fetch(j);
                if (j + 1 < num_kb) {              // past the end: loaded again, not used
                    sx += p.m;
                    ++sw;
                }
            }
            for (int kb0 = 0; kb0 < num_kb; kb0 += C::AHEAD) {
#pragma unroll
                for (int j = 0; j < C::AHEAD; ++j) {
                    const int kb = kb0 + j;
                    if (kb >= num_kb) break;
                    // A wait that ran out ends the tile, not the loop: the warp takes the
                    // remaining groups without waiting or handing buffers back and votes
                    // behind them (a vote per group: 4096x8192x8192 284 us, so 280;
                    // 16 experts of 2048x4096, 4096 tokens 63 us, so 59).
                    ok = ok && mbar_wait_short(&tfull_bar[buf], bphase, &abort_sh, p.status);
                    __syncwarp();
                    tc_fence_after();
                    const float sc = s_a[j] * s_b[j];
                    const float sc2 = C::TWO ? s_a[j] * s_c[C::TWO ? j : 0] : sc;
                    const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * BN + half * C::CW;
#pragma unroll
                    for (int c = 0; c < C::CW / 32; ++c) {
                        uint32_t r[32];
                        tmem_ld32(tb + c * 32, r);
                        tmem_ld_wait();
                        if (c + 1 == C::CW / 32) {
                            // All of this warp's part is in registers: the buffer may be written again.
                            tc_fence_before();
                            if (lane == 0 && ok) mbar_arrive_relaxed(&tempty_bar[buf]);
                        }
                        promote(acc + c * 16, r, C::TWO && c * 32 >= cut ? sc2 : sc);
                    }
                    fetch(j);
                    if (kb + C::AHEAD + 1 < num_kb) {
                        sx += p.m;
                        ++sw;
                    }
                    buf ^= 1;
                    if (buf == 0) bphase ^= 1;
                }
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            // A tensor store clips at the output's last row only: chunks that
            // cross an expert's end are stored row by row.
            const bool tma = use_tmy && (GROUPED ? row0 + 32 <= tr.row_end : row0 < tr.row_end);
#pragma unroll
            for (int c = 0; c < C::CW / 32; ++c) {
                const int n0 = ncol + c * 32;
                if (n0 >= p.n) break;                          // uniform over the warp
                const int nv = (p.n - n0) >= 32 ? 32 : (p.n - n0);   // 16 or 32
                float out[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    out[2 * i] = acc[c * 16 + i].x;
                    out[2 * i + 1] = acc[c * 16 + i].y;
                }
                if (p.bias) {
                    const float4* b4 = reinterpret_cast<const float4*>(p.bias + tr.col_off + n0);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (4 * i >= nv) break;
                        const float4 b = b4[i];
                        out[4 * i] = __fadd_rn(out[4 * i], b.x);
                        out[4 * i + 1] = __fadd_rn(out[4 * i + 1], b.y);
                        out[4 * i + 2] = __fadd_rn(out[4 * i + 2], b.z);
                        out[4 * i + 3] = __fadd_rn(out[4 * i + 3], b.w);
                    }
                }
                if (tma) {
                    uint8_t* b = store;
                    if (lane == 0) bulk_wait_read<0>();        // the previous store has read it
                    __syncwarp();
                    const uint32_t sz = static_cast<uint32_t>((lane >> 1) & 3);   // TMA's 64-byte swizzle
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        st_shared_v4(b + lane * 64 + ((static_cast<uint32_t>(j) ^ sz) << 4),
                                     pack_bf16(out[8 * j], out[8 * j + 1]), pack_bf16(out[8 * j + 2], out[8 * j + 3]),
                                     pack_bf16(out[8 * j + 4], out[8 * j + 5]), pack_bf16(out[8 * j + 6], out[8 * j + 7]));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tmY, b, n0, row0);
                        bulk_commit();
                    }
                } else if (row < tr.row_end) {
                    uint4* yp = reinterpret_cast<uint4*>(p.y + static_cast<int64_t>(row) * p.ldy + n0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (8 * j >= nv) break;
                        yp[j] = make_uint4(pack_bf16(out[8 * j], out[8 * j + 1]), pack_bf16(out[8 * j + 2], out[8 * j + 3]),
                                           pack_bf16(out[8 * j + 4], out[8 * j + 5]), pack_bf16(out[8 * j + 6], out[8 * j + 7]));
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();   // staged output stores done before the CTA ends
        __syncwarp();
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// ============================================================================
// Decode kernel: weights as the MMA's M side, tokens as N, split-K in a cluster
// ============================================================================
//
// 128 output channels and up to NT tokens per cluster; the CTAs of a cluster
// share the K groups and push their fp32 sums, four tokens of a channel at a
// time, to the rank that finishes those tokens, which adds them in rank order.
// A promotion is a chain of about 1000 cycles (barrier, scales, TMEM load,
// sums), longer than an SM's share of the weight stream takes per group.  With
// 32 or 64 tokens two teams of four warps therefore take the groups in turn, each
// with two accumulators and sums of its own (48x14336x4096: 21.3 -> 17.5 us);
// with 128, whose sums would not fit twice, two sets of warps take half the
// columns each; with 16 one team will do, and leaves room for two CTAs per SM.
// With QX the activation arrives unquantized and eight more warps quantize it
// on its way into the stages (the codes are those of the activation
// quantizer): a warp takes four tokens of one K group, and the groups go
// round the warps, since one such piece is a chain of about 1000 cycles too
// (all of a stage's tokens on one warp: 16x14336x4096 16.3 -> 19.6 us).
//   warp 0 TMA, warp 1 MMA, then the promotion warps, then the quantizing ones.

constexpr int kQxWarps = 8;

template <int NT, bool QX>
struct BlockDecodeCfg {
    static constexpr int TEAMS = NT == 32 || NT == 64 ? 2 : 1;
    static constexpr int HALVES = NT == 128 ? 2 : 1;
    static constexpr int SETS = TEAMS * HALVES;  // sets of four promotion warps
    static constexpr int PROMO = 4 * SETS;
    static constexpr int THREADS = 32 * (2 + PROMO + (QX ? kQxWarps : 0));
    static constexpr int CW = NT / HALVES;       // columns per promotion warp
    static constexpr int A_BYTES = kBM * kBKB;   // 128 weight rows
    static constexpr int B_BYTES = NT * kBKB;    // NT token rows
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int MAX_STAGES = NT <= 64 ? 8 : 5;
    // Scales of groups quantized on the way: a stage is refilled when its MMA
    // is done, with the promotion at most four groups behind the MMA.
    static constexpr int SX_RING = MAX_STAGES + 4;
    static constexpr int STATIC = 4 * 1024 + (QX ? 0 : PROMO * kScaleRing * CW * 4);   // static shared memory, at most
    static constexpr int TMEM_COLS = 2 * TEAMS * NT;   // at least the 32 an allocation takes
    static_assert(!QX || (NT == 16 && TEAMS == 1), "the quantizing warps cover 16 tokens and count on one team to free stages");
};

template <int NT, bool QX, typename T>
__global__ void __launch_bounds__(BlockDecodeCfg<NT, QX>::THREADS, 1)
gemm_block_decode_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                         const T* X, int64_t ldx, int k, const BlockParams p, int num_kb,
                         int kb_per_split, int splits, int nstages) {
    using C = BlockDecodeCfg<NT, QX>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    float4* red = reinterpret_cast<float4*>(smem + nstages * C::STAGE);   // [rank][team][quads owned][128 channels]
    __shared__ __align__(8) uint64_t full_bar[C::MAX_STAGES];
    __shared__ __align__(8) uint64_t empty_bar[C::MAX_STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[2 * C::TEAMS];    // [team][accumulator]
    __shared__ __align__(8) uint64_t tempty_bar[2 * C::TEAMS];
    __shared__ __align__(8) uint64_t drain_bar;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    __shared__ __align__(16) float col_s[C::PROMO][C::CW];         // promotion warps: Sx Sw of the group
    __shared__ float sxa_ring[QX ? 1 : C::PROMO][QX ? 1 : kScaleRing][QX ? 1 : C::CW];
    __shared__ float sw_ring[C::PROMO][kScaleRing];
    __shared__ float sx_ring[QX ? C::SX_RING : 1][QX ? NT : 1];
    __shared__ __align__(8) uint64_t sx_bar[QX ? C::SX_RING : 1];  // every quad of the slot is written

    const int warp = warp_index();
    const int lane = threadIdx.x % 32;
    const int tn = blockIdx.x;                       // 128 output channels
    const int t0 = static_cast<int>(blockIdx.z) * NT;
    const int mt = min(NT, p.m - t0);                // this tile's tokens
    const int quads = (mt + 3) / 4;
    const uint32_t rank = cluster_ctarank();         // split index along K
    const int kb0 = static_cast<int>(rank) * kb_per_split;
    const int kb1 = min(num_kb, kb0 + kb_per_split);
    const int my_kb = kb1 > kb0 ? kb1 - kb0 : 0;
    const int qpo = (quads + splits - 1) / splits;   // quads finished per rank

    if (threadIdx.x == 0) {
        for (int s = 0; s < nstages; ++s) {
            mbar_init(&full_bar[s], QX ? 1 + quads : 1);   // TMA (and the quantized quads)
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2 * C::TEAMS; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], C::PROMO / C::TEAMS);
        }
        if constexpr (QX)
            for (int s = 0; s < C::SX_RING; ++s) mbar_init(&sx_bar[s], quads);
        mbar_init(&drain_bar, 1);
        abort_sh = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;
    cluster_started();
    pdl_launch_dependents();

    if (warp == 0) {
        if (elect_one()) {
            constexpr uint32_t kBytes = QX ? C::A_BYTES : C::STAGE;
            tma_prefetch_desc(&tmW);
            if constexpr (!QX) tma_prefetch_desc(&tmX);
            // The weights do not depend on the previous kernel: their first
            // ring goes out before the programmatic-launch wait.
            const int first = my_kb < nstages ? my_kb : nstages;
            for (int i = 0; i < first; ++i) {
                mbar_arrive_expect_tx(&full_bar[i], kBytes);
                tma_load_2d(smem + i * C::STAGE, &tmW, &full_bar[i], (kb0 + i) * kBKB, tn * kBM);
            }
            if constexpr (!QX) {
                pdl_wait();
                for (int i = 0; i < first; ++i)
                    tma_load_2d(smem + i * C::STAGE + C::A_BYTES, &tmX, &full_bar[i], (kb0 + i) * kBKB, t0);
            }
            uint32_t issued = (1u << first) - 1u, last_par = 0;
            int stage = first == nstages ? 0 : first;
            uint32_t phase = first == nstages ? 1u : 0u;
            bool ok = true;
            for (int kb = kb0 + first; kb < kb1; ++kb) {
                if (!mbar_wait_short(&empty_bar[stage], phase ^ 1, &abort_sh, p.status)) {
                    ok = false;
                    break;
                }
                uint8_t* sa = smem + stage * C::STAGE;
                mbar_arrive_expect_tx(&full_bar[stage], kBytes);
                tma_load_2d(sa, &tmW, &full_bar[stage], kb * kBKB, tn * kBM);
                if constexpr (!QX) tma_load_2d(sa + C::A_BYTES, &tmX, &full_bar[stage], kb * kBKB, t0);
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == nstages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok)   // the loads already issued land before the CTA leaves
                for (int s = 0; s < nstages; ++s)
                    if (issued & (1u << s)) mbar_wait(&full_bar[s], (last_par >> s) & 1, nullptr, nullptr);
        }
        __syncwarp();
        cluster_wait_started();
    } else if (warp == 1) {
        {
            const bool leader = elect_one();   // one lane issues, as in the tile kernel
            const uint32_t idesc = make_idesc(1, 0, 0, kBM, static_cast<uint32_t>((mt + 15) / 16 * 16));
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = 0; i < my_kb; ++i) {
                const int n = i / C::TEAMS, buf = i % C::TEAMS * 2 + (n & 1);
                if (!__all_sync(0xffffffffu, mbar_wait_short(&tempty_bar[buf], ((n >> 1) & 1) ^ 1, &abort_sh, p.status) &&
                                             mbar_wait_short(&full_bar[stage], phase, &abort_sh, p.status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_addr(smem + stage * C::STAGE);
                const uint64_t ad = sdesc_kmajor_sw128(sa);
                const uint64_t bd = sdesc_kmajor_sw128(sa + C::A_BYTES);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kBKB / 32; ++ks)
                        mma_issue<kKindF8>(tmem_base + buf * NT, ad + 2 * ks, bd + 2 * ks, idesc, ks != 0);
                    tc_commit(&tfull_bar[buf]);
                }
                __syncwarp();
                if (++stage == nstages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok && leader) {
                tc_commit(&drain_bar);
                mbar_wait(&drain_bar, 0, nullptr, nullptr);
            }
        }
        __syncwarp();
        cluster_wait_started();
    } else if (warp < 2 + C::PROMO) {
        const int q = warp & 3, set = (warp - 2) / 4;
        const int team = C::TEAMS == 2 ? set : 0;
        const int ch = q * 32 + lane;
        const int c0 = C::HALVES == 2 ? set * C::CW : 0; // this warp's first token column
        const int cn = min(C::CW, mt - c0);             // and how many it has (may be none)
        const float* sw = p.sw + static_cast<int64_t>(tn) * num_kb + kb0;
        float* cs = col_s[warp - 2];
        float2 acc[C::CW / 2];
#pragma unroll
        for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        // The scales of a group are asked for kAhead of the team's groups before
        // their use, by asynchronous copies into a ring of each warp.
        const int groups = my_kb > team ? (my_kb - team + C::TEAMS - 1) / C::TEAMS : 0;   // of this team
        auto ask_sw = [&](int n) {
            if (n < groups && lane == 0) cp_async4(&sw_ring[warp - 2][n % kScaleRing], sw + team + n * C::TEAMS);
        };
        auto ask_sx = [&](int n) {
            if constexpr (!QX) {
                if (n < groups) {
#pragma unroll
                    for (int c = 0; c < C::CW; c += 32)
                        if (c + lane < cn)
                            cp_async4(&sxa_ring[warp - 2][n % kScaleRing][c + lane],
                                      p.sx + static_cast<int64_t>(kb0 + team + n * C::TEAMS) * p.m + t0 + c0 + c + lane);
                }
            }
            cp_async_commit();
        };
        for (int n = 0; n < kAhead; ++n) ask_sw(n);     // weights do not depend on the previous kernel
        if constexpr (!QX) pdl_wait();
        for (int n = 0; n < kAhead; ++n) ask_sx(n);
        for (int n = 0; n < groups; ++n) {
            const int i = team + n * C::TEAMS, buf = team * 2 + (n & 1), slot = n % kScaleRing;
            ask_sw(n + kAhead);
            ask_sx(n + kAhead);
            cp_async_wait<kAhead>();
            __syncwarp();
            const float swk = sw_ring[warp - 2][slot];
            if constexpr (QX) {
                if (!__all_sync(0xffffffffu, mbar_wait_short(&sx_bar[i % C::SX_RING], (i / C::SX_RING) & 1, &abort_sh, p.status))) break;
                if (lane < C::CW) cs[lane] = lane < cn ? sx_ring[i % C::SX_RING][lane] * swk : 0.f;
            } else {
#pragma unroll
                for (int c = 0; c < C::CW; c += 32)
                    if (c + lane < C::CW) cs[c + lane] = c + lane < cn ? sxa_ring[warp - 2][slot][c + lane] * swk : 0.f;
            }
            if (!__all_sync(0xffffffffu, mbar_wait_short(&tfull_bar[buf], (n >> 1) & 1, &abort_sh, p.status))) break;
            __syncwarp();
            if (warp - 2 == team * 4 && lane == 0) mbar_arrive(&empty_bar[i % nstages]);   // the MMAs have read the stage
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * NT + c0;
            constexpr int LW = C::CW >= 32 ? 32 : 16;   // columns per TMEM load
#pragma unroll
            for (int c = 0; c < C::CW / LW; ++c) {
                if (c * LW < cn) {
                    uint32_t r[LW];
                    tmem_ld(tb + c * LW, r);
                    tmem_ld_wait();
                    promote(acc + c * (LW / 2), r, cs + c * LW);
                }
            }
            tc_fence_before();
            if (lane == 0) mbar_arrive_relaxed(&tempty_bar[buf]);
        }
        // The other CTAs have long started: nothing is waited for here as a rule.
        __syncwarp();
        cluster_wait_started();
        // Quad g of the tile goes to rank g % splits, slot [rank][team][g / splits][channel].
        const uint32_t dst = smem_addr(red) + ((rank * C::TEAMS + team) * qpo * kBM + ch) * 16u;
        uint32_t owner = static_cast<uint32_t>(c0 / 4 % splits), off = static_cast<uint32_t>(c0 / 4 / splits) * (kBM * 16u);
#pragma unroll
        for (int g = 0; g < C::CW / 4; ++g) {
            if (g * 4 < cn) {
                st_shared_cluster_v4(map_shared_rank(dst + off, owner),
                                     make_float4(acc[2 * g].x, acc[2 * g].y, acc[2 * g + 1].x, acc[2 * g + 1].y));
                if (++owner == static_cast<uint32_t>(splits)) {
                    owner = 0;
                    off += kBM * 16u;
                }
            }
        }
        __syncwarp();
    } else if constexpr (QX) {
        // Piece (group i, quad): 8 lanes per token, 16 values each.  A barrier's
        // parity only tells neighbouring phases apart, so no more warps work than
        // leave a warp's groups at most nstages apart: its last group then showed
        // that groups up to i - 2 * nstages have been read (one thread frees the
        // stages, in their order), and only the use before this one is waited for.
        pdl_wait();
        const int qw = warp - 2 - C::PROMO;
        const int sub = lane & 7, tl = lane / 8;
        const int pieces = my_kb * quads;
        const int warps = min(kQxWarps, nstages * quads);
        auto load = [&](int piece, Eight<T>& lo, Eight<T>& hi) {
            const int t = piece % quads * 4 + tl;
            const int col = (kb0 + piece / quads) * kBlock + sub * 16;
            lo.zero();
            hi.zero();
            if (t < mt && col < k) {
                const T* src = X + static_cast<int64_t>(t0 + t) * ldx + col;
                lo.load(src);
                hi.load(src + 8);
            }
        };
        Eight<T> lo, hi;
        const int first = qw < warps ? qw : pieces;   // the others have nothing to do
        if (first < pieces) load(first, lo, hi);
        for (int piece = first; piece < pieces; piece += warps) {
            const int i = piece / quads, t = piece % quads * 4 + tl;
            float s;
            const uint4 w = quantize16<T>(lo, hi, s);
            if (piece + warps < pieces) load(piece + warps, lo, hi);
            const int stage = i % nstages, use = i / nstages;
            const bool ok = use == 0 || mbar_wait_short(&empty_bar[stage], (use - 1) & 1, &abort_sh, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            st_shared_v4(smem + stage * C::STAGE + C::A_BYTES + t * kBKB + ((sub ^ (t & 7)) << 4), w.x, w.y, w.z, w.w);
            if (sub == 0) sx_ring[i % C::SX_RING][t] = s;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full_bar[stage]);
                mbar_arrive(&sx_bar[i % C::SX_RING]);
            }
        }
        __syncwarp();
        cluster_wait_started();
    }

    // Every rank's pushed sums are visible after this barrier; after it no CTA
    // touches another CTA's shared memory, so each may exit when done.
    __syncthreads();
    cluster_sync();

    if (warp >= 2 && warp < 2 + C::PROMO) {
        const int ch = (warp & 3) * 32 + lane, set = (warp - 2) / 4;
        const int n = tn * kBM + ch;
        if constexpr (QX) pdl_wait();   // Y may still be read by the previous kernel
        if (n < p.n && !abort_sh) {
            const float bias = p.bias ? p.bias[n] : 0.f;
            for (int sl = set, g = static_cast<int>(rank) + set * splits; g < quads; sl += C::SETS, g += C::SETS * splits) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int r = 0; r < splits * C::TEAMS; ++r) {
                    const float4 v = red[(r * qpo + sl) * kBM + ch];
                    s.x = __fadd_rn(s.x, v.x);
                    s.y = __fadd_rn(s.y, v.y);
                    s.z = __fadd_rn(s.z, v.z);
                    s.w = __fadd_rn(s.w, v.w);
                }
                const float o[4] = {s.x, s.y, s.z, s.w};
                __nv_bfloat16* y = p.y + static_cast<int64_t>(t0 + 4 * g) * p.ldy + n;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * g + e < mt) y[e * p.ldy] = __float2bfloat16_rn(p.bias ? __fadd_rn(o[e], bias) : o[e]);
            }
        }
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// ============================================================================
// Host side
// ============================================================================
template <typename T>
cudaError_t act_quant(const BlockQuantArgs& a, cudaStream_t s) {
    constexpr int H = sizeof(T) == 2 ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.rows + kActRows - 1) / kActRows), static_cast<unsigned>((a.k + 256 * H - 1) / (256 * H)), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, act_block_quant_kernel<T, H>, static_cast<const T*>(a.src), a.rows, a.k, a.ld,
                              static_cast<uint8_t*>(a.codes), a.scale);
}

template <typename T>
cudaError_t weight_quant(const BlockQuantArgs& a, cudaStream_t s) {
    const int64_t nb = (a.rows + kBlock - 1) / kBlock, kb = (a.k + kBlock - 1) / kBlock;
    weight_block_quant_kernel<T><<<dim3(static_cast<unsigned>(kb), static_cast<unsigned>(nb), static_cast<unsigned>(a.stack)),
                                   256, 0, s>>>(static_cast<const T*>(a.src), a.rows, a.k, a.ld,
                                                static_cast<uint8_t*>(a.codes), a.scale, nb, kb);
    return cudaGetLastError();
}

BlockParams block_params(const BlockLinearArgs& a) {
    BlockParams p = {};
    p.m = static_cast<int>(a.m);
    p.n = static_cast<int>(a.n);
    p.sx = a.sx;
    p.sw = a.sw;
    p.bias = a.bias;
    p.y = a.y;
    p.ldy = a.ldy;
    p.status = device_status_ptr();
    return p;
}

template <int BN, bool GROUPED>
q8_status run_block_tile(const BlockLinearArgs& a, cudaStream_t s) {
    using C = BlockTileCfg<BN>;
    CUtensorMap tA, tB, tY;
    if (!make_map(&tA, a.x_codes, false, a.k, a.m, a.ldx, kBKB, kBM) ||
        !make_map(&tB, a.w_codes, false, a.k, a.experts * a.n, a.ldw, kBKB, BN))
        return Q8_ERR_CUDA;
    const int use_tmy = make_map_y(&tY, a.y, a.n, a.m, a.ldy) ? 1 : 0;
    if (!use_tmy) tY = tA;
    auto kern = gemm_block_tile_kernel<BN, GROUPED>;
    if (set_smem(kern, C::SMEM) != cudaSuccess) return Q8_ERR_LAUNCH;
    // The warpgroups' register shares come out of what the block launches with:
    // a build that launches with fewer would wait for ever.
    static const bool registers_fit = [&] {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, kern) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        return at.numRegs * kTileThreads >= 128 * kTileRegsLow + 256 * kTileRegsHigh;
    }();
    if (!registers_fit) return Q8_ERR_LAUNCH;
    const int tiles_n = static_cast<int>((a.n + BN - 1) / BN);
    const int tiles_m = static_cast<int>((a.m + kBM - 1) / kBM);
    // Grouped: an upper bound (each expert adds at most one partial row tile);
    // the kernel reads the offsets and walks the actual tiles.
    const int64_t tiles = (tiles_m + (GROUPED ? a.experts : 0)) * tiles_n;
    const int sms = sm_count();
    const int num_kb = static_cast<int>((a.k + kBKB - 1) / kBKB);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < sms ? tiles : sms), 1, 1);
    cfg.blockDim = dim3(kTileThreads, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tA, tB, tY, use_tmy, block_params(a), num_kb, tiles_m, tiles_n, a.offsets,
                           static_cast<int>(a.experts)) != cudaSuccess) {
        cudaGetLastError();
        return Q8_ERR_LAUNCH;
    }
    return Q8_OK;
}

template <int NT, bool QX, typename T>
q8_status run_block_decode(const BlockLinearArgs& a, cudaStream_t s) {
    using C = BlockDecodeCfg<NT, QX>;
    CUtensorMap tW, tX;
    if (!make_map(&tW, a.w_codes, false, a.k, a.n, a.ldw, kBKB, kBM)) return Q8_ERR_CUDA;
    if (QX) tX = tW;
    else if (!make_map(&tX, a.x_codes, false, a.k, a.m, a.ldx, kBKB, NT)) return Q8_ERR_CUDA;
    auto kern = gemm_block_decode_kernel<NT, QX, T>;
    const int tiles_n = static_cast<int>((a.n + kBM - 1) / kBM);
    const int tiles_t = static_cast<int>((a.m + NT - 1) / NT);
    const int num_kb = static_cast<int>((a.k + kBKB - 1) / kBKB);
    // Split K across the CTAs of a cluster (at most 8, every split non-empty)
    // as far as one wave holds: two CTAs per SM up to 16 tokens (a short stage
    // ring; with more the registers allow one), and about 128 SMs where clusters
    // of four and eight fit.
    const int per_sm = NT == 16 ? 2 : 1;
    int want = 128 * per_sm / (tiles_n * tiles_t);
    if (want < 1) want = 1;
    if (want > 8) want = 8;
    if (want > num_kb) want = num_kb;
    const int per = (num_kb + want - 1) / want;
    const int splits = (num_kb + per - 1) / per;
    const int quads = ((a.m < NT ? static_cast<int>(a.m) : NT) + 3) / 4;
    const int red = splits * C::TEAMS * ((quads + splits - 1) / splits) * kBM * 16;
    const int budget = (NT == 16 && static_cast<int64_t>(tiles_n) * splits > sm_count() ? 113 : 222) * 1024 - C::STATIC - red;
    int nstages = budget / C::STAGE;
    if (nstages > C::MAX_STAGES) nstages = C::MAX_STAGES;
    if (nstages > per) nstages = per;
    if (nstages < 1) nstages = 1;
    const int smem = nstages * C::STAGE + red + 1024;
    if (set_smem(kern, smem) != cudaSuccess) return Q8_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles_n), static_cast<unsigned>(splits), static_cast<unsigned>(tiles_t));
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tW, tX, static_cast<const T*>(a.x), a.ldx, static_cast<int>(a.k),
                           block_params(a), num_kb, per, splits, nstages) != cudaSuccess) {
        cudaGetLastError();
        return Q8_ERR_LAUNCH;
    }
    return Q8_OK;
}

// Tile width: the persistent grid's makespan, waves x (BN + a tile's fixed cost
// of about 64 columns' worth), the narrower tile on ties.
template <bool GROUPED>
q8_status run_tiles(const BlockLinearArgs& a, int64_t row_tiles, cudaStream_t s) {
    const int64_t sms = sm_count();
    auto cost = [&](int64_t bn) {
        const int64_t tiles = row_tiles * ((a.n + bn - 1) / bn);
        return ((tiles + sms - 1) / sms) * (bn + 64);
    };
    const int64_t narrow = cost(128), middle = cost(192), wide = cost(256);
    if (wide < middle && wide < narrow) return run_block_tile<256, GROUPED>(a, s);
    if (middle < narrow) return run_block_tile<192, GROUPED>(a, s);
    return run_block_tile<128, GROUPED>(a, s);
}

}  // namespace

cudaError_t launch_block_quant(const BlockQuantArgs& a, bool weight, cudaStream_t s) {
    switch (a.src_dtype) {
        case Q8_F16: return weight ? weight_quant<__half>(a, s) : act_quant<__half>(a, s);
        case Q8_BF16: return weight ? weight_quant<__nv_bfloat16>(a, s) : act_quant<__nv_bfloat16>(a, s);
        default: return weight ? weight_quant<float>(a, s) : act_quant<float>(a, s);
    }
}

q8_status launch_block_linear(const BlockLinearArgs& a, cudaStream_t s) {
    if (a.offsets) {
        // Row tiles, estimated: half a partial tile per expert on top of the
        // full ones, and one for every expert where they average fewer rows.
        const int64_t full = (a.m + kBM - 1) / kBM, some = a.experts < a.m ? a.experts : a.m;
        const int64_t rows = full + a.experts / 2 > some ? full + a.experts / 2 : some;
        return run_tiles<true>(a, rows, s);
    }
    if (a.x) {   // quantized on the way
        switch (a.x_dtype) {
            case Q8_F16: return run_block_decode<16, true, __half>(a, s);
            case Q8_BF16: return run_block_decode<16, true, __nv_bfloat16>(a, s);
            default: return run_block_decode<16, true, float>(a, s);
        }
    }
    if (a.m <= 16) return run_block_decode<16, false, __half>(a, s);
    if (a.m <= 32) return run_block_decode<32, false, __half>(a, s);
    // From 33 tokens on the decode GEMM serves where K can be split in one wave
    // (twice up to 64 tokens, four times up to 256); with more output the tile
    // kernel's larger tiles are faster (64x8192x4096: 11.4 us split, 12.6 in tiles;
    // 48x14336x4096: 16.1 and 14.5; 128x4096x4096: 10.1 and 12.3; 256x4096x4096:
    // 15.3 and 12.9; 200x14336x4096: 49 and 21).
    const int64_t tiles_n = (a.n + kBM - 1) / kBM;
    if (a.m <= 64 && tiles_n <= 64) return run_block_decode<64, false, __half>(a, s);
    if (a.m > 64 && a.m <= 2 * kBM && (a.m + kBM - 1) / kBM * tiles_n <= 32)
        return run_block_decode<128, false, __half>(a, s);
    return run_tiles<false>(a, (a.m + kBM - 1) / kBM, s);
}

}  // namespace q8
