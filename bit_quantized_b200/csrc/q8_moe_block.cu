// The expert layer of a mixture of experts for a few tokens, on block-scaled
// FP8 weights, and the router's choice.
//
//   route   the top_k largest logits of a token (the lowest index first among
//           equals), weighted by a softmax or a sigmoid
//   layer   G, U = W13[e] q(x_t),  h = q(silu(G) * U),
//           y_t = sum over the token's experts e of w[t, e] W2[e] h
//           with q the quantizer of one scale per token and 128 values
//
// For a few tokens the layer is the stream of the chosen experts' weights, so
// both projections divide that stream evenly: the K groups of all active
// experts' 128-channel tiles form one line of steps, and every CTA takes an
// equal, contiguous piece of it (weights on the MMA's M side, tokens as N).
// Where a piece ends inside a tile, the fp32 sums go to the workspace, and the
// CTA that arrives last adds them in the order of the CTAs, so results repeat
// bit for bit.  Three launches:
//   moe_prepare_kernel  quantizes x once, lists the active experts with their
//                       tokens, and clears the arrival counters;
//   moe_up_kernel       gate and up tiles side by side, SwiGLU and the
//                       quantization of h in the epilogue (a tile is 128 wide:
//                       one scale group of h);
//   moe_down_kernel     goes through the experts of an output tile one after
//                       the other, so the weighted sum over experts stays in
//                       the CTA's shared memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "q8_block.cuh"
#include "q8_internal.h"
#include "q8_tile.cuh"

namespace q8 {
namespace {

constexpr int kBM = 128;
constexpr int kBKB = 128;
constexpr int kMaxTokens = kMoeMaxTokens;
constexpr int kMaxExperts = kMoeMaxExperts;
constexpr int kMinSteps = 4;   // fewest K groups worth a CTA of its own

// ============================================================================
// Router
// ============================================================================
//
// One warp per token, 16 logits per lane.  A logit becomes an ordered 32-bit
// key (0: not to be chosen), so a round of the selection is one warp maximum
// and, for the lowest index among equals, one warp minimum.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0u;                   // -inf and NaN are never chosen
    v = fminf(v, FLT_MAX) + 0.0f;                      // -0 equals 0
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__global__ void __launch_bounds__(128)
moe_route_kernel(const T* logits, int64_t ld, int64_t m, int experts, int top_k, int sigmoid,
                 int renormalize, int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int lane = threadIdx.x % 32;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
    pdl_wait();
    pdl_launch_dependents();
    if (t >= m) return;
    constexpr int V = kMaxExperts / 32;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        key[i] = e < experts ? order_key(to_float(logits[t * ld + e])) : 0u;
    }
    uint32_t lead = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) lead = max(lead, key[i]);
    lead = __reduce_max_sync(0xffffffffu, lead);
    const float top = lead ? key_value(lead) : 0.f;
    float total = 0.f;
    if (!sigmoid && !renormalize) {                    // softmax over all experts
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i]) total += expf(key_value(key[i]) - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    int my_id = -1;                                    // lane s: slot s
    float my_w = 0.f;
    for (int s = 0; s < top_k; ++s) {
        uint32_t best = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == 0u) break;
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (key[i] == best) at = static_cast<uint32_t>(i * 32 + lane);
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (static_cast<uint32_t>(i * 32 + lane) == at) key[i] = 0u;
        if (lane == s) {
            my_id = static_cast<int>(at);
            const float v = key_value(best);
            my_w = sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - top);
        }
    }
    if (renormalize) {
        total = my_w;
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane < top_k) {
        if (renormalize || !sigmoid) my_w = total > 0.f ? my_w / total : 0.f;
        ids[t * top_k + lane] = my_id;
        weights[t * top_k + lane] = my_w;
    }
}

// ============================================================================
// Preparation: x in 8 bits, the active experts, cleared counters
// ============================================================================

struct MoeParams {
    int m, top_k, experts, hidden, inter;
    int rows_max;            // m * top_k
    int it, ht, kb1, kb2;    // 128-wide tiles of inter and hidden; K groups of both products (kb1 = ht, kb2 = it)
    int* head;               // [0] active experts
    int* expert;             // [active] expert of each active index, ascending
    int* base;               // [active + 1] first row of its tokens; a row is a (token, expert) pair
    int* row_token;          // [rows] an expert's tokens, ascending
    float* row_weight;       // [rows]
    int* up_count; int* down_count;
    uint8_t* xq; float* xs;  // m x hidden codes, [kb1][m]
    uint8_t* hq; float* hs;  // rows x inter codes, [kb2][rows_max]
    float* part;             // sums of unfinished tiles
    const float* s13; const float* s2;
    __nv_bfloat16* y; int64_t ldy;
    int* status;
};

template <typename T>
__global__ void __launch_bounds__(256)
moe_prepare_kernel(const T* X, int64_t ldx, const int32_t* ids, const float* weights, const MoeParams p) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (blockIdx.x > 0) {
        // 256 columns (two groups) of eight tokens, a warp each.
        const int cols = (p.hidden + 255) / 256;
        const int col = (static_cast<int>(blockIdx.x) - 1) % cols * 256 + lane * 8;
        const int t = (static_cast<int>(blockIdx.x) - 1) / cols * 8 + warp;
        pdl_wait();
        pdl_launch_dependents();
        if (t >= p.m) return;
        Eight<T> v;
        if (col < p.hidden) v.load(X + static_cast<int64_t>(t) * ldx + col);
        else v.zero();
        float f[8];
        v.values(f);
        float a = v.absmax();
#pragma unroll
        for (int o = 8; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const BlockScale s = block_scale(a);
        if (col < p.hidden) {
            *reinterpret_cast<uint2*>(p.xq + static_cast<int64_t>(t) * p.hidden + col) =
                make_uint2(block_codes4(f[0], f[1], f[2], f[3], s), block_codes4(f[4], f[5], f[6], f[7], s));
            if (lane % 16 == 0) p.xs[static_cast<int64_t>(col / kBlock) * p.m + t] = s.S;
        }
        return;
    }
    // The first block: tokens of every expert as a bit mask (an expert that a
    // token names twice has it once, with both weights), then the list.
    __shared__ unsigned long long mask_sh[kMaxExperts];
    __shared__ int base_sh[kMaxExperts];                 // by expert: its first row
    __shared__ int ids_sh[kMaxTokens * kMoeMaxTopK];
    __shared__ float weights_sh[kMaxTokens * kMoeMaxTopK];
    for (int e = threadIdx.x; e < p.experts; e += 256) mask_sh[e] = 0ull;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < p.rows_max; i += 256) {
        const int e = ids[i];
        ids_sh[i] = e;
        weights_sh[i] = weights[i];
        if (e >= 0 && e < p.experts) atomicOr(&mask_sh[e], 1ull << (i / p.top_k));
    }
    for (int i = threadIdx.x; i < min(p.experts, p.rows_max) * p.it; i += 256) p.up_count[i] = 0;
    for (int i = threadIdx.x; i < p.ht; i += 256) p.down_count[i] = 0;
    __syncthreads();
    if (warp == 0) {
        int na = 0, nr = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < p.experts ? __popcll(mask_sh[e]) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (c > 0) {
                const int a = na + __popc(some & ((1u << lane) - 1u));
                p.expert[a] = e;
                p.base[a] = base_sh[e] = nr + incl - c;
            }
            na += __popc(some);
            nr += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            p.head[0] = na;
            p.base[na] = nr;
        }
    }
    __syncthreads();
    // A thread per choice: the first of a token's choices of an expert writes the row.
    for (int i = threadIdx.x; i < p.rows_max; i += 256) {
        const int e = ids_sh[i], t = i / p.top_k;
        if (e < 0 || e >= p.experts) continue;
        bool again = false;
        float w = 0.f;
        for (int s = t * p.top_k; s < (t + 1) * p.top_k; ++s)
            if (ids_sh[s] == e) {
                if (s < i) again = true;
                w += weights_sh[s];
            }
        if (again) continue;
        const int r = base_sh[e] + __popcll(mask_sh[e] & ((1ull << t) - 1ull));
        p.row_token[r] = t;
        p.row_weight[r] = w;
    }
}

// ============================================================================
// The two products
// ============================================================================
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A CTA's piece of the line of steps, and which CTA a step belongs to.
struct Line {
    long long total;
    int ctas;
    __device__ __forceinline__ Line(long long t) : total(t) {
        long long c = t / kMinSteps;
        ctas = static_cast<int>(c < 1 ? 1 : (c < static_cast<long long>(gridDim.x) ? c : static_cast<long long>(gridDim.x)));
    }
    __device__ __forceinline__ int start(int c) const { return static_cast<int>(total * c / ctas); }
    __device__ __forceinline__ int owner(int s) const {
        return static_cast<int>(((static_cast<long long>(s) + 1) * ctas - 1) / total);
    }
};

// The tiles of a CTA's steps [begin, end) in the order it takes them: the piece
// of the tile that the next CTA goes on with first, then the piece of the tile
// that an earlier CTA began, then the whole tiles, so that the wait for other
// contributors' sums lies under the whole tiles' stream.
struct Pieces {
    int begin, end, steps, first, count;
    bool tail;
    __device__ __forceinline__ Pieces(int b, int e, int steps_per_tile) : begin(b), end(e), steps(steps_per_tile) {
        first = b / steps_per_tile;
        count = b < e ? (e - 1) / steps_per_tile - first + 1 : 0;
        tail = e % steps_per_tile != 0;
    }
    __device__ __forceinline__ int tile(int i) const { return tail ? (i == 0 ? first + count - 1 : first + i - 1) : first + i; }
    __device__ __forceinline__ int k0(int u) const { return max(begin - u * steps, 0); }
    __device__ __forceinline__ int k1(int u) const { return min(end - u * steps, steps); }
};

// The expert list in shared memory, copied by the whole block in one round
// trip: every entry there may be is read, what lies past the active ones is not
// used.
struct ListSh {
    int active;
    int expert[kMaxExperts];
    int base[kMaxExperts + 1];
};

__device__ __forceinline__ void copy_list(ListSh& l, uint8_t* token_sh, const MoeParams& p) {
    const int most = min(p.experts, p.rows_max);
    if (threadIdx.x == 0) l.active = __ldcg(p.head);
    for (int a = threadIdx.x; a <= most; a += blockDim.x) {
        if (a < most) l.expert[a] = __ldcg(p.expert + a);
        l.base[a] = __ldcg(p.base + a);
    }
    if (token_sh)
        for (int r = threadIdx.x; r < p.rows_max; r += blockDim.x) token_sh[r] = static_cast<uint8_t>(__ldcg(p.row_token + r));
    __syncthreads();
}

// Counts this CTA's arrival at a tile with `parts` contributors; true in the
// one that arrives last, which then sees every contributor's sums.  Called by
// 128 threads after each wrote its sums; the leader's fences cover them all
// (the barriers order the others' accesses before and after).
__device__ __forceinline__ bool arrive_last(int* counter, int parts, int* flag_sh, bool leader, int barrier) {
    named_barrier(barrier, 128);
    if (leader) {
        __threadfence();
        *flag_sh = atomicAdd(counter, 1) == parts - 1;
        __threadfence();
    }
    named_barrier(barrier, 128);
    const bool last = *flag_sh != 0;
    named_barrier(barrier, 128);   // the flag may be written again
    return last;
}

template <int NT>
struct MoeUpCfg {
    // Two teams of four promotion warps take the tiles in turn: one finishes a
    // tile (SwiGLU, scales and codes of h) while the other promotes the next.
    // Each has two accumulators and barriers of its own: a barrier's parity
    // only tells neighbouring phases apart.
    static constexpr int THREADS = 32 * (2 + 8);
    static constexpr int B_BYTES = NT * kBKB;
    static constexpr int STAGE = 2 * kBM * kBKB + B_BYTES;
    // About 100 KB of weights on their way per SM: a longer ring streams no
    // faster and only delays what waits behind it, the sums that contributors
    // exchange (64 tokens over 32 experts of 2880 x 1408: 98 us with three
    // stages, 101 with four).
    static constexpr int STAGES = 3;
    static constexpr int TMEM_COLS = 8 * NT;
    static constexpr int SMEM = STAGES * STAGE + 1024;
};

template <int NT>
__global__ void __launch_bounds__(MoeUpCfg<NT>::THREADS, 1)
moe_up_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const MoeParams p) {
    using C = MoeUpCfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    __shared__ __align__(8) uint64_t full_bar[C::STAGES];
    __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[4];    // [team][accumulator]
    __shared__ __align__(8) uint64_t tempty_bar[4];
    __shared__ __align__(8) uint64_t drain_bar;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh, last_sh[2];
    __shared__ __align__(16) float col_s[8][2][NT];
    __shared__ float amax_sh[2][4][NT];
    __shared__ float sx_ring[8][kScaleRing][NT], sw_ring[8][kScaleRing][2];
    __shared__ ListSh list;
    __shared__ uint8_t token_sh[kMaxTokens * kMoeMaxTopK];

    const int warp = warp_index(), lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], 4);
        }
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
    pdl_wait();
    // The down projection may start: it reads the expert list, which is
    // complete here, before it waits for this kernel.
    pdl_launch_dependents();

    copy_list(list, token_sh, p);
    const int active = list.active;
    const Line line(static_cast<long long>(active) * p.it * p.kb1);
    const int cta = static_cast<int>(blockIdx.x);
    const int s_begin = active > 0 && cta < line.ctas ? line.start(cta) : 0;
    const int s_end = active > 0 && cta < line.ctas ? line.start(cta + 1) : 0;
    const Pieces pieces(s_begin, s_end, p.kb1);

    if (warp == 0) {
        if (elect_one() && s_begin < s_end) {
            tma_prefetch_desc(&tmW);
            tma_prefetch_desc(&tmX);
            uint32_t issued = 0, last_par = 0;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = 0; i < pieces.count && ok; ++i) {
                const int u = pieces.tile(i), k0 = pieces.k0(u), k1 = pieces.k1(u);
                const int a = u / p.it;
                const int row = list.expert[a] * 2 * p.inter + (u - a * p.it) * kBM;
                const int base = list.base[a], cnt = list.base[a + 1] - base;
                const int quads = (cnt + 3) / 4;
                for (int kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait_short(&empty_bar[stage], phase ^ 1, &abort_sh, p.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = smem + stage * C::STAGE;
                    mbar_arrive_expect_tx(&full_bar[stage], 2 * kBM * kBKB + quads * 4 * kBKB);
                    tma_load_2d(sa, &tmW, &full_bar[stage], kb * kBKB, row);
                    tma_load_2d(sa + kBM * kBKB, &tmW, &full_bar[stage], kb * kBKB, row + p.inter);
                    // The expert's tokens, four rows of x at a time (the last one again past the end).
                    for (int b = 0; b < quads; ++b) {
                        const uint8_t* tk = token_sh + base + 4 * b;
                        const int last = cnt - 1 - 4 * b;
                        tma_gather4(sa + (2 * kBM + 4 * b) * kBKB, &tmX, &full_bar[stage], kb * kBKB, tk[0],
                                    tk[min(1, last)], tk[min(2, last)], tk[min(3, last)]);
                    }
                    issued |= 1u << stage;
                    last_par = (last_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok)   // the loads already issued land before the CTA leaves
                for (int t = 0; t < C::STAGES; ++t)
                    if (issued & (1u << t)) mbar_wait(&full_bar[t], (last_par >> t) & 1, nullptr, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        {
            // The whole warp runs the loop and one lane issues: descriptors then
            // stay in uniform registers.
            const bool leader = elect_one();
            int stage = 0;
            uint32_t phase = 0;
            int n_even = 0, n_odd = 0;                     // steps of team 0 and of team 1
            bool ok = true;
            for (int i = 0; i < pieces.count && ok; ++i) {
                const int u = pieces.tile(i), k0 = pieces.k0(u), k1 = pieces.k1(u);
                const int a = u / p.it, team = i & 1;
                const int cnt = list.base[a + 1] - list.base[a];
                const uint32_t idesc = make_idesc(1, 0, 0, kBM, static_cast<uint32_t>((cnt + 15) / 16 * 16));
                int n = team ? n_odd : n_even;
                for (int kb = k0; kb < k1; ++kb, ++n) {
                    const int buf = team * 2 + (n & 1);
                    if (!__all_sync(0xffffffffu, mbar_wait_short(&tempty_bar[buf], ((n >> 1) & 1) ^ 1, &abort_sh, p.status) &&
                                                 mbar_wait_short(&full_bar[stage], phase, &abort_sh, p.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + stage * C::STAGE);
                    const uint64_t gd = sdesc_kmajor_sw128(sa), ud = sdesc_kmajor_sw128(sa + kBM * kBKB);
                    const uint64_t bd = sdesc_kmajor_sw128(sa + 2 * kBM * kBKB);
                    const uint32_t d = tmem_base + buf * 2 * NT;
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < kBKB / 32; ++ks) {
                            mma_issue<kKindF8>(d, gd + 2 * ks, bd + 2 * ks, idesc, ks != 0);
                            mma_issue<kKindF8>(d + NT, ud + 2 * ks, bd + 2 * ks, idesc, ks != 0);
                        }
                        tc_commit(&tfull_bar[buf]);
                        tc_commit(&empty_bar[stage]);
                    }
                    __syncwarp();
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (team) n_odd = n;
                else n_even = n;
            }
            if (!ok && leader) {
                tc_commit(&drain_bar);
                mbar_wait(&drain_bar, 0, nullptr, nullptr);
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, team = (warp - 2) / 4;
        const int ch = q * 32 + lane;
        const bool lead = (warp - 2) % 4 == 0 && lane == 0;
        float* cs = &col_s[warp - 2][0][0];
        constexpr int NS = (NT + 31) / 32;
        // The team's step whose scales are asked for next.
        int ai = team, akb = 0, aend = 0, acn = 0, asked = 0, used = 0;
        int atok[NS];
        const float* asw = nullptr;
        auto enter = [&] {                                  // its tile
            const int au = pieces.tile(ai), a = au / p.it, base = list.base[a];
            acn = list.base[a + 1] - base;
#pragma unroll
            for (int c = 0; c < NS; ++c) atok[c] = c * 32 + lane < acn ? token_sh[base + c * 32 + lane] : 0;
            akb = pieces.k0(au);
            aend = pieces.k1(au);
            asw = p.s13 + (static_cast<int64_t>(list.expert[a]) * 2 * p.it + (au - a * p.it)) * p.kb1;
        };
        auto ask = [&] {
            if (ai < pieces.count) {
                const int slot = asked++ % kScaleRing;
#pragma unroll
                for (int c = 0; c < NS; ++c)
                    if (c * 32 + lane < acn)
                        cp_async4(&sx_ring[warp - 2][slot][c * 32 + lane], p.xs + static_cast<int64_t>(akb) * p.m + atok[c]);
                if (lane < 2) cp_async4(&sw_ring[warp - 2][slot][lane], asw + static_cast<int64_t>(lane) * p.it * p.kb1 + akb);
                if (++akb == aend) {                        // the next tile is the other team's
                    ai += 2;
                    if (ai < pieces.count) enter();
                }
            }
            cp_async_commit();
        };
        if (ai < pieces.count) enter();
        for (int i = 0; i < kAhead; ++i) ask();
        // After a wait that ran out, the warps stop waiting and reading TMEM but
        // take the same barriers to the end (the status word tells the caller).
        bool ok = true;
        for (int i = team; i < pieces.count; i += 2) {
            const int u = pieces.tile(i), k0 = pieces.k0(u), k1 = pieces.k1(u);
            const int a = u / p.it, it = u - a * p.it;
            const int row0 = list.base[a], cn = list.base[a + 1] - row0;   // column i is row row0 + i
            float2 g[NT / 2], w[NT / 2];
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) g[i] = w[i] = make_float2(0.f, 0.f);
            for (int kb = k0; kb < k1; ++kb) {
                ask();
                cp_async_wait<kAhead>();
                __syncwarp();
                const int slot = used % kScaleRing;
#pragma unroll
                for (int c = 0; c < NS; ++c) {
                    const int i = c * 32 + lane;
                    if (i < NT) {
                        const float sx = sx_ring[warp - 2][slot][i];
                        cs[i] = sx * sw_ring[warp - 2][slot][0];
                        cs[NT + i] = sx * sw_ring[warp - 2][slot][1];
                    }
                }
                const int buf = team * 2 + (used & 1);
                ok = ok && mbar_wait_short(&tfull_bar[buf], (used >> 1) & 1, &abort_sh, p.status);
                ++used;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                __syncwarp();                               // every lane's columns of cs (a vote orders no memory)
                tc_fence_after();
                const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * 2 * NT;
#pragma unroll
                for (int c = 0; c < NT / 16; ++c) {
                    if (c * 16 < cn) {
                        uint32_t rg[16], ru[16];
                        tmem_ld16(tb + c * 16, rg);
                        tmem_ld16(tb + NT + c * 16, ru);
                        tmem_ld_wait();
                        promote(g + c * 8, rg, cs + c * 16);
                        promote(w + c * 8, ru, cs + NT + c * 16);
                    }
                }
                tc_fence_before();
                if (lane == 0) mbar_arrive_relaxed(&tempty_bar[buf]);
            }
            // From here on the sums are in local memory, so that loops over the
            // tokens need not be unrolled: unrolled, this part is tens of KB of
            // code, and its instructions come from HBM while the weights stream
            // through L2 (64 tokens: 36 us per tile against 2).
            float tg[NT], tw[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i < cn) {
                    tg[i] = (i & 1) ? g[i / 2].y : g[i / 2].x;
                    tw[i] = (i & 1) ? w[i / 2].y : w[i / 2].x;
                }
            bool finish = true;
            if (k1 - k0 < p.kb1) {
                // A piece of a tile: [cta][first or last tile][gate, up][column][channel].
                float* mine = p.part + (static_cast<int64_t>(cta) * 2 + (k0 > 0 ? 0 : 1)) * (2 * NT * kBM) + ch;
#pragma unroll 1
                for (int i = 0; i < cn; ++i) {
                    mine[i * kBM] = tg[i];
                    mine[(NT + i) * kBM] = tw[i];
                }
                const int first = line.owner(u * p.kb1), lastc = line.owner((u + 1) * p.kb1 - 1);
                finish = arrive_last(&p.up_count[u], lastc - first + 1, &last_sh[team], lead, 1 + team);
                if (finish) {
                    // Four contributors' sums of two tokens are asked for together.
                    auto part = [&](int c) {
                        return p.part + (static_cast<int64_t>(c) * 2 + (c > first ? 0 : 1)) * (2 * NT * kBM) + ch;
                    };
#pragma unroll 1
                    for (int i = 0; i < cn; i += 2) {
                        const int i1 = min(i + 1, cn - 1);
                        float g0 = 0.f, g1 = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll 1
                        for (int c = first; c <= lastc; c += 4) {
                            float x[4][4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float* src = part(min(c + j, lastc));
                                x[j][0] = __ldcg(src + i * kBM);
                                x[j][1] = __ldcg(src + i1 * kBM);
                                x[j][2] = __ldcg(src + (NT + i) * kBM);
                                x[j][3] = __ldcg(src + (NT + i1) * kBM);
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (c + j <= lastc) {
                                    g0 += x[j][0];
                                    g1 += x[j][1];
                                    w0 += x[j][2];
                                    w1 += x[j][3];
                                }
                        }
                        tg[i1] = g1;
                        tw[i1] = w1;
                        tg[i] = i1 > i ? g0 : g1;
                        tw[i] = i1 > i ? w0 : w1;
                    }
                }
            }
            if (finish) {
                // h = silu(G) U of this tile: one scale group of h per token.
#pragma unroll 1
                for (int i = 0; i < cn; i += 2) {
                    const int i1 = min(i + 1, cn - 1);
                    const float g0 = tg[i], g1 = tg[i1];
                    const float h0 = g0 / (1.0f + expf(-g0)) * tw[i], h1 = g1 / (1.0f + expf(-g1)) * tw[i1];
                    const uint32_t m0 = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(h0)));
                    const uint32_t m1 = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(h1)));
                    if (lane == 0) {
                        amax_sh[team][q][i] = __uint_as_float(m0);
                        amax_sh[team][q][i1] = __uint_as_float(m1);
                    }
                    tg[i] = h0;
                    if (i1 > i) tg[i1] = h1;
                }
                named_barrier(3 + team, 128);
                // A lane computes a token's scale; the others take it from there.
#pragma unroll 1
                for (int i0 = 0; i0 < cn; i0 += 32) {
                    const int il = min(i0 + lane, NT - 1);
                    const BlockScale bs = block_scale(fmaxf(fmaxf(amax_sh[team][0][il], amax_sh[team][1][il]),
                                                            fmaxf(amax_sh[team][2][il], amax_sh[team][3][il])));
                    if (q == 0 && i0 + lane < cn) p.hs[static_cast<int64_t>(it) * p.rows_max + row0 + i0 + lane] = bs.S;
#pragma unroll 2
                    for (int i = i0; i < min(cn, i0 + 32); ++i) {
                        BlockScale b;
                        b.S = __shfl_sync(0xffffffffu, bs.S, i - i0);
                        b.R = __shfl_sync(0xffffffffu, bs.R, i - i0);
                        b.Rlo = __shfl_sync(0xffffffffu, bs.Rlo, i - i0);
                        p.hq[static_cast<int64_t>(row0 + i) * p.inter + it * kBM + ch] =
                            static_cast<uint8_t>(block_codes4(tg[i], 0.f, 0.f, 0.f, b) & 0xFFu);
                    }
                }
                named_barrier(3 + team, 128);   // amax_sh may be written again
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

template <int NT>
struct MoeDownCfg {
    static constexpr int THREADS = 32 * (2 + 8);      // four promotion warps, four that only help to sum
    static constexpr int B_BYTES = NT * kBKB;
    static constexpr int STAGE = kBM * kBKB + B_BYTES;
    static constexpr int OUT = NT * kBM * 4;          // the tile's sums over experts
    static constexpr int STAGES = NT <= 32 ? 7 : 5;   // about 100 KB of weights, as above
    static constexpr int TMEM_COLS = 2 * NT;
    static constexpr int SUM_TOKENS = 4;              // tokens a warp sums at a time
    static constexpr int SMEM = STAGES * STAGE + OUT + 1024;
};

template <int NT>
__global__ void __launch_bounds__(MoeDownCfg<NT>::THREADS, 1)
moe_down_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH, const MoeParams p) {
    using C = MoeDownCfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    float* out = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);   // [token][channel]
    __shared__ __align__(8) uint64_t full_bar[C::STAGES];
    __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[2];
    __shared__ __align__(8) uint64_t tempty_bar[2];
    __shared__ __align__(8) uint64_t drain_bar;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh, last_sh, sum_sh[3];   // sum_sh: whether to sum, over which CTAs
    __shared__ __align__(16) float col_s[4][NT];
    __shared__ float sh_ring[4][kScaleRing][NT], sw_ring[4][kScaleRing];
    __shared__ ListSh list;

    const int warp = warp_index(), lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], 4);
        }
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
    pdl_launch_dependents();

    // The expert list was complete before the up projection let this kernel start.
    copy_list(list, nullptr, p);
    const int active = list.active;
    const int tile_steps = active * p.kb2;           // of one output tile
    const Line line(static_cast<long long>(tile_steps) * p.ht);
    const int cta = static_cast<int>(blockIdx.x);
    const int s_begin = active > 0 && cta < line.ctas ? line.start(cta) : 0;
    const int s_end = active > 0 && cta < line.ctas ? line.start(cta + 1) : 0;

    // The finished rows of an output tile, four channels per lane and a token
    // per warp: the sums over experts, or those of all contributors in the order
    // of the CTAs.
    auto sum_tile = [&](int nt, int first, int lastc) {
        const int n = nt * kBM + lane * 4;
#pragma unroll 1
        for (int t = warp - 2; t < p.m; t += 8 * C::SUM_TOKENS) {
            float4 v[C::SUM_TOKENS];
#pragma unroll
            for (int j = 0; j < C::SUM_TOKENS; ++j) {
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (first == lastc && t + 8 * j < p.m)
                    v[j] = *reinterpret_cast<const float4*>(out + (t + 8 * j) * kBM + lane * 4);
            }
            if (first != lastc) {
#pragma unroll 4
                for (int c = first; c <= lastc; ++c) {
                    const float* src = p.part + (static_cast<int64_t>(c) * 2 + (c > first ? 0 : 1)) * (p.m * kBM) + lane * 4;
#pragma unroll
                    for (int j = 0; j < C::SUM_TOKENS; ++j) {
                        const float4 x = __ldcg(reinterpret_cast<const float4*>(src + min(t + 8 * j, p.m - 1) * kBM));
                        v[j].x += x.x;
                        v[j].y += x.y;
                        v[j].z += x.z;
                        v[j].w += x.w;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < C::SUM_TOKENS; ++j)
                if (t + 8 * j < p.m && n < p.hidden)
                    *reinterpret_cast<uint2*>(p.y + static_cast<int64_t>(t + 8 * j) * p.ldy + n) =
                        make_uint2(pack_bf16(v[j].x, v[j].y), pack_bf16(v[j].z, v[j].w));
        }
    };

    if (warp == 0) {
        if (elect_one() && s_begin < s_end) {
            tma_prefetch_desc(&tmW);
            tma_prefetch_desc(&tmH);
            uint32_t issued = 0, last_par = 0;
            bool ok = true;
            // Pass 0 asks for the first ring's weights without waiting for the up
            // projection, pass 1 for everything else.  An SM holds no CTA of both
            // projections (registers, shared memory, with 64 tokens TMEM too), so this
            // one starts when an up CTA has left, and the head start is the time from
            // there to the end of the last up CTA.
            const int first = min(s_end - s_begin, C::STAGES);
            for (int pass = 0; pass < 2 && ok; ++pass) {
                if (pass == 1) pdl_wait();
                int stage = 0;
                uint32_t phase = 0;
                const int end = pass == 0 ? s_begin + first : s_end;
                for (int s = s_begin; s < end && ok;) {
                    const int v = s / p.kb2, k0 = s - v * p.kb2;
                    const int k1 = min(p.kb2, k0 + end - s);
                    const int nt = v / active, a = v - nt * active;
                    const int row = list.expert[a] * p.hidden + nt * kBM;
                    const int base = list.base[a];
                    const int boxes = (list.base[a + 1] - base + 15) / 16;
                    for (int kb = k0; kb < k1; ++kb, ++s) {
                        const bool early = s - s_begin < first;
                        uint8_t* sa = smem + stage * C::STAGE;
                        if (pass == 1 && !early && !mbar_wait_short(&empty_bar[stage], phase ^ 1, &abort_sh, p.status)) {
                            ok = false;
                            break;
                        }
                        if (pass == 0 || !early) {
                            mbar_arrive_expect_tx(&full_bar[stage], kBM * kBKB + boxes * 16 * kBKB);
                            tma_load_2d(sa, &tmW, &full_bar[stage], kb * kBKB, row);
                            issued |= 1u << stage;
                            last_par = (last_par & ~(1u << stage)) | (phase << stage);
                        }
                        if (pass == 1)
                            for (int b = 0; b < boxes; ++b)
                                tma_load_2d(sa + kBM * kBKB + b * 16 * kBKB, &tmH, &full_bar[stage], kb * kBKB, base + b * 16);
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
            }
            if (!ok)
                for (int t = 0; t < C::STAGES; ++t)
                    if (issued & (1u << t)) mbar_wait(&full_bar[t], (last_par >> t) & 1, nullptr, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        {
            const bool leader = elect_one();
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true;
            for (int s = s_begin; s < s_end && ok;) {
                const int v = s / p.kb2, k0 = s - v * p.kb2;
                const int k1 = min(p.kb2, k0 + s_end - s);
                const int a = v % active;
                const int cnt = list.base[a + 1] - list.base[a];
                const uint32_t idesc = make_idesc(1, 0, 0, kBM, static_cast<uint32_t>((cnt + 15) / 16 * 16));
                for (int kb = k0; kb < k1; ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait_short(&tempty_bar[buf], bphase ^ 1, &abort_sh, p.status) &&
                                                 mbar_wait_short(&full_bar[stage], phase, &abort_sh, p.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + stage * C::STAGE);
                    const uint64_t ad = sdesc_kmajor_sw128(sa), bd = sdesc_kmajor_sw128(sa + kBM * kBKB);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < kBKB / 32; ++ks)
                            mma_issue<kKindF8>(tmem_base + buf * NT, ad + 2 * ks, bd + 2 * ks, idesc, ks != 0);
                        tc_commit(&tfull_bar[buf]);
                        tc_commit(&empty_bar[stage]);
                    }
                    __syncwarp();
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                    buf ^= 1;
                    if (buf == 0) bphase ^= 1;
                }
                s += k1 - k0;
            }
            if (!ok && leader) {
                tc_commit(&drain_bar);
                mbar_wait(&drain_bar, 0, nullptr, nullptr);
            }
        }
        __syncwarp();
    } else if (warp >= 6) {
        // The helpers of the sums over contributors.
        pdl_wait();
        for (int s = s_begin; s < s_end;) {
            const int nt = s / tile_steps;
            named_barrier(2, 256);
            if (sum_sh[0]) sum_tile(nt, sum_sh[1], sum_sh[2]);
            named_barrier(2, 256);
            s = min((nt + 1) * tile_steps, s_end);
        }
    } else {
        pdl_wait();
        const int q = warp & 3;
        const int ch = q * 32 + lane;
        float* cs = col_s[q];
        // The step whose scales are asked for next.
        int as = s_begin, akb = 0, ant = 0, aa = 0, abase = 0, acnt = 0;
        const float* asw = nullptr;
        if (s_begin < s_end) {
            const int v0 = s_begin / p.kb2;
            akb = s_begin - v0 * p.kb2;
            ant = v0 / active;
            aa = v0 - ant * active;
        }
        auto enter = [&] {                                  // its expert
            abase = list.base[aa];
            acnt = list.base[aa + 1] - abase;
            asw = p.s2 + (static_cast<int64_t>(list.expert[aa]) * p.ht + ant) * p.kb2;
        };
        auto ask = [&] {
            if (as < s_end) {
                const int slot = (as - s_begin) % kScaleRing;
#pragma unroll
                for (int c = 0; c < NT; c += 32)
                    if (c + lane < acnt)
                        cp_async4(&sh_ring[q][slot][c + lane], p.hs + static_cast<int64_t>(akb) * p.rows_max + abase + c + lane);
                if (lane == 0) cp_async4(&sw_ring[q][slot], asw + akb);
                ++as;
                if (++akb == p.kb2) {
                    akb = 0;
                    if (++aa == active) {
                        aa = 0;
                        ++ant;
                    }
                    if (as < s_end) enter();
                }
            }
            cp_async_commit();
        };
        if (s_begin < s_end) enter();
        for (int i = 0; i < kAhead; ++i) ask();
        float* oc = out + ch;
        if (active == 0) {                           // no token chose an expert: y is zero
            for (int nt = cta; nt < p.ht; nt += static_cast<int>(gridDim.x))
                if (nt * kBM + ch < p.hidden)
                    for (int t = 0; t < p.m; ++t) p.y[t * p.ldy + nt * kBM + ch] = __float2bfloat16_rn(0.f);
        }
        int buf = 0;
        uint32_t bphase = 0;
        bool ok = true;   // as in the up projection
        for (int s = s_begin; s < s_end;) {
            // One output tile, or this CTA's piece of it.
            const int nt = s / tile_steps;
            const int tile0 = nt * tile_steps, tile1 = tile0 + tile_steps;
            const int s0 = s, s1 = min(tile1, s_end);
            for (int t = 0; t < p.m; ++t) oc[t * kBM] = 0.f;
            while (s < s1) {
                const int v = s / p.kb2, k0 = s - v * p.kb2;
                const int k1 = min(p.kb2, k0 + s1 - s);
                const int a = v - nt * active;
                const int base = list.base[a], cnt = list.base[a + 1] - base;
                float2 acc[NT / 2];
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
                constexpr int NS = (NT + 31) / 32;
                int tk[NS];                      // the rows' tokens and weights, one row per lane
                float wt[NS];
#pragma unroll
                for (int c = 0; c < NS; ++c) {
                    const bool have = c * 32 + lane < cnt;
                    tk[c] = have ? __ldcg(p.row_token + base + c * 32 + lane) : 0;
                    wt[c] = have ? __ldcg(p.row_weight + base + c * 32 + lane) : 0.f;
                }
                for (int kb = k0; kb < k1; ++kb) {
                    ask();
                    cp_async_wait<kAhead>();
                    __syncwarp();
                    const int slot = (s + kb - k0 - s_begin) % kScaleRing;
#pragma unroll
                    for (int c = 0; c < NS; ++c)
                        if (c * 32 + lane < NT) cs[c * 32 + lane] = sh_ring[q][slot][c * 32 + lane] * sw_ring[q][slot];
                    ok = ok && mbar_wait_short(&tfull_bar[buf], bphase, &abort_sh, p.status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    __syncwarp();                // every lane's columns of cs (a vote orders no memory)
                    tc_fence_after();
                    const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * NT;
#pragma unroll
                    for (int c = 0; c < NT / 16; ++c) {
                        if (c * 16 < cnt) {
                            uint32_t r[16];
                            tmem_ld16(tb + c * 16, r);
                            tmem_ld_wait();
                            promote(acc + c * 8, r, cs + c * 16);
                        }
                    }
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_relaxed(&tempty_bar[buf]);
                    buf ^= 1;
                    if (buf == 0) bphase ^= 1;
                }
                // The expert's weighted rows join the tile's sums (a thread owns its
                // channel); its tokens differ, so four are loaded together.  In
                // local memory and rolled, as in the up projection.
                float ta[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    if (i < cnt) ta[i] = (i & 1) ? acc[i / 2].y : acc[i / 2].x;
#pragma unroll 1
                for (int i0 = 0; i0 < cnt; i0 += 4) {
                    int at[4];
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = min(i0 + e, cnt - 1);
                        const bool high = NT > 32 && i >= 32;
                        at[e] = __shfl_sync(0xffffffffu, high ? tk[NS - 1] : tk[0], i % 32) * kBM;
                        const float wi = __shfl_sync(0xffffffffu, high ? wt[NS - 1] : wt[0], i % 32);
                        v[e] = __fmaf_rn(wi, ta[i], oc[at[e]]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i0 + e < cnt) oc[at[e]] = v[e];
                }
                s += k1 - k0;
            }
            bool finish = true;
            int first = cta, lastc = cta;
            if (s1 - s0 < tile_steps) {
                float* mine = p.part + (static_cast<int64_t>(cta) * 2 + (s0 > tile0 ? 0 : 1)) * (p.m * kBM) + ch;
                for (int t = 0; t < p.m; ++t) mine[t * kBM] = oc[t * kBM];
                first = line.owner(tile0);
                lastc = line.owner(tile1 - 1);
                finish = arrive_last(&p.down_count[nt], lastc - first + 1, &last_sh, warp == 2 && lane == 0, 1);
            }
            if (warp == 2 && lane == 0) {
                sum_sh[0] = finish;
                sum_sh[1] = first;
                sum_sh[2] = lastc;
            }
            named_barrier(2, 256);                   // every channel's sums are in shared memory
            if (finish) sum_tile(nt, first, lastc);
            named_barrier(2, 256);                   // before the sums of the next tile
        }
        __syncwarp();
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
cudaError_t route(const MoeRouteArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.m + 3) / 4), 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_route_kernel<T>, static_cast<const T*>(a.logits), a.ld, a.m,
                              static_cast<int>(a.experts), static_cast<int>(a.top_k), a.sigmoid ? 1 : 0,
                              a.renormalize ? 1 : 0, a.ids, a.weights);
}

// The workspace, cut up in this order; returns its size (base may be null).
int64_t layout(const MoeLayerArgs& a, uint8_t* base, MoeParams* p) {
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    const int64_t rows = a.m * a.top_k, act = a.experts < rows ? a.experts : rows;
    const int64_t it = a.inter / kBlock, ht = (a.hidden + kBlock - 1) / kBlock;
    const int64_t nt = a.m <= 16 ? 16 : a.m <= 32 ? 32 : 64;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t* r = base + at;
        at += up(bytes);
        return r;
    };
    uint8_t* head = take(8);
    uint8_t* expert = take(4 * act);
    uint8_t* first = take(4 * (act + 1));
    uint8_t* token = take(4 * rows);
    uint8_t* weight = take(4 * rows);
    uint8_t* upc = take(4 * act * it);
    uint8_t* downc = take(4 * ht);
    uint8_t* xq = take(a.m * a.hidden);
    uint8_t* xs = take(4 * a.m * ht);
    uint8_t* hq = take(rows * a.inter);
    uint8_t* hs = take(4 * rows * it);
    // The up projection's sums are dead before the down projection writes its own.
    const int64_t part_up = 4 * 2 * nt * kBM, part_down = 4 * a.m * kBM;
    uint8_t* part = take(2 * kMoeMaxCtas * (part_up > part_down ? part_up : part_down));
    if (p) {
        p->m = static_cast<int>(a.m);
        p->top_k = static_cast<int>(a.top_k);
        p->experts = static_cast<int>(a.experts);
        p->hidden = static_cast<int>(a.hidden);
        p->inter = static_cast<int>(a.inter);
        p->rows_max = static_cast<int>(rows);
        p->it = p->kb2 = static_cast<int>(it);
        p->ht = p->kb1 = static_cast<int>(ht);
        p->head = reinterpret_cast<int*>(head);
        p->expert = reinterpret_cast<int*>(expert);
        p->base = reinterpret_cast<int*>(first);
        p->row_token = reinterpret_cast<int*>(token);
        p->row_weight = reinterpret_cast<float*>(weight);
        p->up_count = reinterpret_cast<int*>(upc);
        p->down_count = reinterpret_cast<int*>(downc);
        p->xq = xq;
        p->xs = reinterpret_cast<float*>(xs);
        p->hq = hq;
        p->hs = reinterpret_cast<float*>(hs);
        p->part = reinterpret_cast<float*>(part);
        p->s13 = a.s13;
        p->s2 = a.s2;
        p->y = a.y;
        p->ldy = a.ldy;
        p->status = device_status_ptr();
    }
    return at;
}

template <typename K, typename... Args>
q8_status launch(K kern, int blocks, int threads, int smem, cudaStream_t s, Args... args) {
    if (smem > 0 && set_smem(kern, smem) != cudaSuccess) return Q8_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return Q8_ERR_LAUNCH;
    }
    return Q8_OK;
}

template <typename T>
q8_status prepare(const MoeLayerArgs& a, const MoeParams& p, cudaStream_t s) {
    return launch(moe_prepare_kernel<T>, static_cast<int>((a.hidden + 255) / 256 * ((a.m + 7) / 8)) + 1, 256, 0, s,
                  static_cast<const T*>(a.x), a.ldx, a.ids, a.weights, p);
}

template <int NT>
q8_status products(const MoeLayerArgs& a, const MoeParams& p, cudaStream_t s) {
    CUtensorMap tW13, tX, tW2, tH;
    if (!make_map(&tW13, a.w13, false, a.hidden, a.experts * 2 * a.inter, a.ld13, kBKB, kBM) ||
        !make_map(&tX, p.xq, false, a.hidden, a.m, a.hidden, kBKB, 1) ||
        !make_map(&tW2, a.w2, false, a.inter, a.experts * a.hidden, a.ld2, kBKB, kBM) ||
        !make_map(&tH, p.hq, false, a.inter, p.rows_max, a.inter, kBKB, 16))
        return Q8_ERR_CUDA;
    const int ctas = sm_count() < kMoeMaxCtas ? sm_count() : static_cast<int>(kMoeMaxCtas);
    const q8_status st = launch(moe_up_kernel<NT>, ctas, MoeUpCfg<NT>::THREADS, MoeUpCfg<NT>::SMEM, s, tW13, tX, p);
    if (st != Q8_OK) return st;
    using D = MoeDownCfg<NT>;
    return launch(moe_down_kernel<NT>, ctas, D::THREADS, D::SMEM, s, tW2, tH, p);
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t s) {
    switch (a.dtype) {
        case Q8_F16: return route<__half>(a, s);
        case Q8_BF16: return route<__nv_bfloat16>(a, s);
        default: return route<float>(a, s);
    }
}

int64_t moe_workspace_bytes(const MoeLayerArgs& a) { return layout(a, nullptr, nullptr); }

q8_status launch_moe_layer(const MoeLayerArgs& a, uint8_t* workspace, cudaStream_t s) {
    MoeParams p = {};
    layout(a, workspace, &p);
    q8_status st;
    switch (a.x_dtype) {
        case Q8_F16: st = prepare<__half>(a, p, s); break;
        case Q8_BF16: st = prepare<__nv_bfloat16>(a, p, s); break;
        default: st = prepare<float>(a, p, s); break;
    }
    if (st != Q8_OK) return st;
    if (a.m <= 16) return products<16>(a, p, s);
    if (a.m <= 32) return products<32>(a, p, s);
    return products<64>(a, p, s);
}

}  // namespace q8
