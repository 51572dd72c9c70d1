// qnn_gemv.cuh -- what the kernels of qgemv_w4 share: the arguments, the conversion of
// codes to the tensor cores' operand, the parts of fp32 x, the loads of weights.
#pragma once
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>
#include "qnn_float.cuh"
#include "qnn_internal.h"
#include "qnn_ptx.cuh"

namespace qnn {

struct GemvArgs {
    const void *x;
    const uint8_t *w;
    const uint8_t *scale;  // [tile][G][8][2] of scale_dt
    const uint8_t *zero;   // [tile][G][8][2], or nullptr
    const float *bias;
    void *y;
    int64_t ldx, ldy, M;
    int N, K, tiles, steps, groups;
    int per_scale;   // how many of a step's NS scales a group lasts
    int y_dt, scale_dt;
    int align;       // bytes, 16 at most, on whose multiples the rows of x start
    int sets;        // of the channels that a block has at a time
    uint32_t *status;  // device status word
};

// The product for more columns of x than the eight of one mma.sync tile.
qnn_status launch_gemv_columns(const GemvArgs &a, int x_dt, int group, cudaStream_t s);

// (w & mask) | magic in one logic operation
__device__ __forceinline__ uint32_t nib(uint32_t w, uint32_t mask, uint32_t magic)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t fma2_u32(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The zero points of a lane's two channels as the addends of the code conversion.
// f16: 0x6400 | q is 1024 + q, and 0x6400 | 16 q is 1024 + 16 q, which a multiply by
// 1/16 takes to 64 + q.  bf16: 0x4300 | q is 128 + q (the nibbles shifted down, as
// 128 + 16 q would not fit its 8 bits).  Subtracting magic + z is exact: |q - z| <= 15.
struct ZeroTerm {
    uint32_t lo, hi;
};

template <bool BF16>
__device__ __forceinline__ ZeroTerm zero_term(uint32_t z_lo, uint32_t z_hi)
{
    if constexpr (BF16) return {0xc300c300u + z_lo * 0x10001u, 0xc300c300u + z_hi * 0x10001u};
    return {0xe400e400u + z_lo * 0x10001u, 0xd400d400u + z_hi * 0x100010u};
}

template <bool BF16>
__device__ __forceinline__ void codes_to_a(uint32_t w, const ZeroTerm &z, uint32_t (&a)[4])
{
    if constexpr (BF16) {
        const uint32_t one = 0x3f803f80u;
        a[0] = fma2_u32<true>(nib(w, 0x000f000fu, 0x43004300u), one, z.lo);
        a[1] = fma2_u32<true>(nib(w >> 4, 0x000f000fu, 0x43004300u), one, z.hi);
        a[2] = fma2_u32<true>(nib(w >> 8, 0x000f000fu, 0x43004300u), one, z.lo);
        a[3] = fma2_u32<true>(nib(w >> 12, 0x000f000fu, 0x43004300u), one, z.hi);
    } else {
        const uint32_t one = 0x3c003c00u, sixteenth = 0x2c002c00u, v = w >> 8;
        a[0] = fma2_u32<false>(nib(w, 0x000f000fu, 0x64006400u), one, z.lo);
        a[1] = fma2_u32<false>(nib(w, 0x00f000f0u, 0x64006400u), sixteenth, z.hi);
        a[2] = fma2_u32<false>(nib(v, 0x000f000fu, 0x64006400u), one, z.lo);
        a[3] = fma2_u32<false>(nib(v, 0x00f000f0u, 0x64006400u), sixteenth, z.hi);
    }
}

// Column of the B operand -> (row of x, part).  fp32 rows take three columns: x is the
// exact sum of three bf16, its leading 8 bits, the next 8 and the rest, each cut (not
// rounded, so that none overflows); infinities and NaN go into the first alone.
template <int XT>
struct Cols {
    static constexpr int kParts = XT == QNN_F32 ? 3 : 1;
};

// columns of the B operand that one pass over the weights takes at most
constexpr int kMaxCols = 32;

__device__ __forceinline__ void bf16_parts(float v, uint32_t (&p)[3])
{
    const uint32_t u = __float_as_uint(v);
    p[0] = u >> 16;
    p[1] = p[2] = 0;
    if ((u & 0x7f800000u) == 0x7f800000u) {
        if (u & 0x007fffffu) p[0] = 0x7fc0u;
        return;
    }
    const float r1 = __fsub_rn(v, __uint_as_float(u & 0xffff0000u));  // exact, as is r2
    p[1] = __float_as_uint(r1) >> 16;
    const float r2 = __fsub_rn(r1, __uint_as_float(p[1] << 16));
    p[2] = __float_as_uint(r2) >> 16;
}

// Global loads that stay behind grid_dependency_wait.  The grid before may write what they read
// while this one has already begun, so that it is no constant of this grid (__ldg).
__device__ __forceinline__ uint32_t load_input(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint16_t load_input(const uint16_t *p)
{
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ float load_input(const float *p)
{
    return __uint_as_float(load_input(reinterpret_cast<const uint32_t *>(p)));
}

__device__ __forceinline__ uint2 load_input(const uint2 *p)
{
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 load_input(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// One scale as it is kept, and its value: apart, so that nothing waits for the load.
__device__ __forceinline__ uint32_t load_scale(const uint8_t *p, int dt, int64_t i)
{
    return dt == QNN_F32 ? load_input(reinterpret_cast<const uint32_t *>(p) + i)
                         : (uint32_t)load_input(reinterpret_cast<const uint16_t *>(p) + i);
}

__device__ __forceinline__ float scale_f32(uint32_t s, int dt)
{
    if (dt == QNN_F32) return __uint_as_float(s);
    return dt == QNN_F16 ? __half2float(__ushort_as_half((uint16_t)s)) : __uint_as_float(s << 16);
}

__device__ __forceinline__ void store_y(const GemvArgs &a, int64_t at, float v)
{
    if (a.y_dt == QNN_F32) static_cast<float *>(a.y)[at] = v;
    else if (a.y_dt == QNN_F16) static_cast<__half *>(a.y)[at] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16 *>(a.y)[at] = from_f32<__nv_bfloat16>(v);
}

// A lane's two scales as they are kept: fp32 in both words, 16-bit types in the first.
__device__ __forceinline__ uint2 load_scales(const uint8_t *p, int dt)
{
    return dt == QNN_F32 ? load_input(reinterpret_cast<const uint2 *>(p))
                         : make_uint2(load_input(reinterpret_cast<const uint32_t *>(p)), 0u);
}

__device__ __forceinline__ float2 scales_f32(uint2 s, int dt)
{
    if (dt == QNN_F32) return make_float2(__uint_as_float(s.x), __uint_as_float(s.y));
    if (dt == QNN_BF16) return make_float2(__uint_as_float(s.x << 16), __uint_as_float(s.x & 0xffff0000u));
    __half2 h;
    memcpy(&h, &s.x, 4);
    return __half22float2(h);
}

// 32 bytes read once
__device__ __forceinline__ void ldg_stream_v8(const uint8_t *p, uint32_t (&w)[8])
{
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

// `bytes` (a multiple of 16) from p, 16-byte aligned, into L2
__device__ __forceinline__ void prefetch_l2(const void *p, int bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

}  // namespace qnn
