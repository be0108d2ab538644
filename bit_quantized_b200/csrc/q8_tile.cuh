// What the tcgen05 GEMM kernels share: the persistent schedules' tile maps
// (dense, and grouped by expert), and the host side of a launch (tensor maps,
// the shared-memory limit, how many CTAs or CTA pairs the device holds).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "q8_device.cuh"
#include "q8_smem.h"

namespace q8 {
namespace {

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// bf16_rne(a) in the low half, bf16_rne(b) in the high half (one conversion).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void st_shared_v4(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr(p)), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Where one output tile of a persistent schedule lies.
struct TileRef {
    int a_row;     // first activation row the tile reads
    int row_end;   // rows at or past row_end are computed and not stored
    int b_row;     // first weight row
    int n_tile;    // first output column
    int col_off;   // offset of the output columns in the scale and bias arrays
};

// Dense schedule: tiles_m x tiles_n tiles, the M index fastest.
__device__ __forceinline__ TileRef dense_tile(int tile, int tiles_m, int rows, int bn, int m) {
    const int tm = tile % tiles_m, tn = tile / tiles_m;
    return TileRef{tm * rows, m, tn * bn, tn * bn, 0};
}

// Grouped schedule of a mixture-of-experts layer (the grouped FP8 linear of
// the FBGEMM FP8 page, section 5.4): tokens sorted by expert, rows
// off[e] .. off[e+1]-1 meet expert e's weight rows e*n .. e*n+n-1.  Expert e
// has ceil((off[e+1] - off[e]) / rows) row tiles; mt[e] counts those of the
// experts before it, so the layer has mt[E] x tiles_n tiles, the row-tile index
// fastest.  A tile starts at any token row (TMA has no alignment rule for the
// outer coordinate); rows past the expert's end are computed and not stored.
constexpr int kMaxGroupedExperts = 512;

__device__ __forceinline__ TileRef grouped_tile(int tile, const int* off, const int* mt, int experts,
                                                int rows, int bn, int n) {
    const int G = mt[experts];
    const int g = tile % G, tn = tile / G;
    // the expert e with mt[e] <= g < mt[e + 1] (empty experts have none)
    int lo = 0, hi = experts;   // mt[lo] <= g < mt[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (mt[mid] <= g) lo = mid; else hi = mid;
    }
    return TileRef{off[lo] + (g - mt[lo]) * rows, off[lo + 1], lo * n + tn * bn, tn * bn, lo * n};
}

// off[0..E]: the offsets clamped to [0, m] and made non-decreasing; mt[0..E]:
// the row-tile prefix.  One warp, 32 experts at a time.
__device__ __forceinline__ void build_group_map(const int32_t* offsets, int experts, int m, int rows,
                                                int* off, int* mt) {
    const int lane = threadIdx.x % 32;
    int carry_off = 0, carry_mt = 0;
    for (int base = 0; base <= experts; base += 32) {
        const int e = base + lane;
        int v = e <= experts ? offsets[e] : m;
        v = v < 0 ? 0 : (v > m ? m : v);
        v = v > carry_off ? v : carry_off;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {   // running maximum
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = v > y ? v : y;
        }
        // expert e - 1 spans [off[e - 1], off[e]): its row tiles, counted at index e
        const int prev = __shfl_up_sync(0xffffffffu, v, 1);
        const int lo_e = lane == 0 ? carry_off : prev;
        int t = (e >= 1 && e <= experts) ? (v - lo_e + rows - 1) / rows : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {   // inclusive sum
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        if (e <= experts) {
            off[e] = v;
            mt[e] = carry_mt + t;
        }
        carry_off = __shfl_sync(0xffffffffu, v, 31);
        carry_mt += __shfl_sync(0xffffffffu, t, 31);
    }
}

// ---------------------------------------------------------------- host side

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2-D K-major tile map with 128-byte swizzle: inner extent `inner` elements of
// `esize` bytes, `outer` rows `ld_bytes` apart, box of (box_inner, box_outer).
inline bool make_map(CUtensorMap* m, const void* base, bool fp16, uint64_t inner, uint64_t outer,
              uint64_t ld_bytes, uint32_t box_inner, uint32_t box_outer) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {ld_bytes};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of the bf16 output for the epilogue's staged stores: boxes of
// 32 columns x 32 rows with the 64-byte swizzle of the staging buffers.
inline bool make_map_y(CUtensorMap* m, const void* y, uint64_t n, uint64_t rows, uint64_t ldy_elems) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {n, rows};
    const cuuint64_t strides[1] = {ldy_elems * 2};
    const cuuint32_t box[2] = {32, 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(y), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int sm_count() {
    static int cached[64] = {0};
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return n;
    }
    if (cached[dev] > 0) return cached[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    cached[dev] = n;
    return n;
}

// Pairs that fit on the device at once (clusters of two 1-CTA-per-SM CTAs),
// cached per kernel instantiation and device.
template <typename K>
int max_pairs(K kernel, int smem, int threads) {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sm_count() / 2;
    if (cached[dev] > 0) return cached[dev];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = sm_count() / 2;
    }
    cached[dev] = n;
    return n;
}

}  // namespace
}  // namespace q8
