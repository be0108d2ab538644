// Device pieces of the block-scaled FP8 format, shared by the quantizers, the
// GEMMs and the expert layer: one scale per 128 values,
//   S = max(fl32(absmax / 448), 1e-8),  q = e4m3_rne_satfinite(fl32(x / S)),
// with the IEEE quotient reached without a division per element
// (q8_qmath.cuh), so every kernel that quantizes gives the same codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "q8_device.cuh"
#include "q8_qmath.cuh"

namespace q8 {
namespace {

constexpr int kBlock = 128;   // values per scale along K, rows per weight scale

// Where K groups are short, their scales are asked for kAhead groups before
// their use, by asynchronous copies into a ring of each promotion warp (a
// weight's scale comes from memory, and a group takes a few hundred cycles).
constexpr int kAhead = 6, kScaleRing = 8;

struct BlockScale {
    float S, R, Rlo;
};

__device__ __forceinline__ BlockScale block_scale(float amax) {
    BlockScale b;
    b.S = __fdiv_rn(amax, 448.0f);
    if (!(b.S >= qm::kEps)) b.S = qm::kEps;
    b.R = __frcp_rn(b.S);
    b.Rlo = qm::reciprocal_low(b.S, b.R);
    return b;
}

// Codes of four values.  |x / S| is at most 448 (1 + 2^-24) and S at least
// 1e-8, inside quotient2's domain.  The quotient of -0 comes out as +0, so each
// code takes its value's sign.
__device__ __forceinline__ uint32_t block_codes4(float a, float b, float c, float d, const BlockScale& s) {
    const float2 nS = make_float2(-s.S, -s.S), R = make_float2(s.R, s.R), L = make_float2(s.Rlo, s.Rlo);
    const float2 q0 = qm::quotient2(make_float2(a, b), nS, R, L);
    const float2 q1 = qm::quotient2(make_float2(c, d), nS, R, L);
    const uint32_t c0 = __nv_cvt_float2_to_fp8x2(q0, __NV_SATFINITE, __NV_E4M3);
    const uint32_t c1 = __nv_cvt_float2_to_fp8x2(q1, __NV_SATFINITE, __NV_E4M3);
    const uint32_t sg = __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0073),
                                    __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0073), 0x5410);
    return __byte_perm(c0, c1, 0x5410) | (sg & 0x80808080u);
}

__device__ __forceinline__ void widen2(uint32_t u, float& a, float& b, __nv_bfloat16) {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xFFFF0000u);
}

__device__ __forceinline__ void widen2(uint32_t u, float& a, float& b, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    a = f.x;
    b = f.y;
}

// Largest magnitude of 8 16-bit values, two at a time (exact: a maximum rounds
// nothing).
__device__ __forceinline__ float pair_max(__nv_bfloat162 a) { return fmaxf(__low2float(a), __high2float(a)); }
__device__ __forceinline__ float pair_max(__half2 a) { return fmaxf(__low2float(a), __high2float(a)); }

template <typename T2>
__device__ __forceinline__ float absmax8_pairs(uint4 u) {
    const uint32_t w[4] = {u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu, u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu};
    const T2* h = reinterpret_cast<const T2*>(w);
    return pair_max(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
}

__device__ __forceinline__ float absmax8_16(uint4 u, __nv_bfloat16) { return absmax8_pairs<__nv_bfloat162>(u); }
__device__ __forceinline__ float absmax8_16(uint4 u, __half) { return absmax8_pairs<__half2>(u); }

// 8 consecutive values as fp32, from a 16-byte-aligned address.  Plain loads:
// with programmatic launch the previous kernel may write its output while this
// one is already resident, so nothing it wrote is read as constant data.
template <typename T>
struct Eight {
    uint4 u;
    __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float absmax() const { return absmax8_16(u, T()); }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        widen2(u.x, f[0], f[1], T());
        widen2(u.y, f[2], f[3], T());
        widen2(u.z, f[4], f[5], T());
        widen2(u.w, f[6], f[7], T());
    }
};

template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float absmax() const {
        return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                     fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// Scales of the tile kernel's promotion.  Volatile keeps the loads where they
// stand.  An activation's may be written by the previous kernel while this one
// is resident, so they are read by ordinary loads behind the programmatic-launch
// wait.  A weight's are complete before this kernel starts (the launch-overlap
// rule of the interface) and stay as they are: read-only data.
__device__ __forceinline__ float ld_act_scale(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ float ld_weight_scale(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// One quantization group spread over 8 lanes (16 values each): codes of this
// lane's 16 values and the group's scale.
template <typename T>
__device__ __forceinline__ uint4 quantize16(const Eight<T>& lo, const Eight<T>& hi, float& scale) {
    float a[8], b[8];
    lo.values(a);
    hi.values(b);
    float m = fmaxf(lo.absmax(), hi.absmax());
#pragma unroll
    for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale s = block_scale(m);
    scale = s.S;
    return make_uint4(block_codes4(a[0], a[1], a[2], a[3], s), block_codes4(a[4], a[5], a[6], a[7], s),
                      block_codes4(b[0], b[1], b[2], b[3], s), block_codes4(b[4], b[5], b[6], b[7], s));
}

// acc[i] += s * part[i] for 32 accumulator columns in registers, with one
// scale.  Volatile, so that the additions stay before the next tensor-memory
// load: moved behind it, they keep both loads' registers alive and spill.
__device__ __forceinline__ void promote(float2* acc, const uint32_t (&r)[32], float s) {
    unsigned long long s2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
#pragma unroll
    for (int i = 0; i < 16; ++i)
        asm volatile(
            "{\n\t.reg .b64 p, a;\n\t"
            "mov.b64 p, {%2, %3};\n\t"
            "mov.b64 a, {%0, %1};\n\t"
            "fma.rn.f32x2 a, p, %4, a;\n\t"
            "mov.b64 {%0, %1}, a;\n\t}"
            : "+f"(acc[i].x), "+f"(acc[i].y)
            : "r"(r[2 * i]), "r"(r[2 * i + 1]), "l"(s2));
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }

// The same for N columns with a scale per column, from 16-byte-aligned shared memory.
template <int N>
__device__ __forceinline__ void promote(float2* acc, const uint32_t (&r)[N], const float* s) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(s + 4 * i);
        acc[2 * i] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])),
                                make_float2(v.x, v.y), acc[2 * i]);
        acc[2 * i + 1] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                                    make_float2(v.z, v.w), acc[2 * i + 1]);
    }
}

}  // namespace
}  // namespace q8
