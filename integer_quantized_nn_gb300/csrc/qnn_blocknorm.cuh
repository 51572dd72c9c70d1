// qnn_blocknorm.cuh -- what q_block_norm and q_block_norm_backward share: rows of the
// float types in registers, their reductions and statistics, argument checks and launch.
#pragma once
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>
#include "qnn_float.cuh"
#include "qnn_internal.h"
#include "qnn_ptx.cuh"

namespace qnn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxC = 32768;
constexpr int kMaxStages = 4;
// Shared memory of an SM given to rings: what covers the latency twice over; the rest
// stays L1, which holds the parameters.
constexpr int kRingSmem = 128 << 10;
constexpr int kRingCarveout = 60;  // percent of the SM's memory
constexpr int kMaxRing = 200 << 10;  // a single block's ring at most
constexpr int kMaxRingC = 8192;      // columns of the rows that go through rings, at most

// V consecutive elements as fp32 (V = 8: 16-byte accesses; V = 1: any address)
template <int V, typename T>
__device__ __forceinline__ void load_v(const T *p, float *v)
{
    if constexpr (V == 1) {
        v[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        T t[8];
        memcpy(t, &u, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
    }
}

template <int V, typename T>
__device__ __forceinline__ void store_v(T *p, const float *v)
{
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *(reinterpret_cast<float4 *>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(v[i]);
        uint4 u;
        memcpy(&u, t, 16);
        *reinterpret_cast<uint4 *>(p) = u;
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t as_u64(float2 v)
{
    uint64_t u;
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(v.x), "f"(v.y));
    return u;
}

__device__ __forceinline__ float2 as_f2(uint64_t u)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(u));
    return v;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_f2(d);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(d);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Two sums at once: the half-warps take one each, after exchanging what the other needs;
// lanes 0 .. 15 get v.x's, 16 .. 31 v.y's.
__device__ __forceinline__ float half_sums(float2 v)
{
    const bool upper = threadIdx.x & 16;
    float s = upper ? v.y : v.x;
    s += __shfl_xor_sync(kFull, upper ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    return s;
}

// Sums (or maxima) over a row's threads: a warp, or the block through shared memory.
// Two slots used in turn make one barrier per call enough: a slot is written again
// only behind the barrier that follows its last read.
struct RowReduce {
    float (*slots)[64];
    int turn = 0;

    template <bool WARP>
    __device__ __forceinline__ float2 sum(float2 v)
    {
        float s = half_sums(v);
        const int lane = threadIdx.x & 31, l = lane & 15, at = (lane >> 4) * 32;
        if constexpr (!WARP) {
            float *slot = slots[turn];
            turn ^= 1;
            const int warps = blockDim.x >> 5;
            if (l == 0) slot[at + (threadIdx.x >> 5)] = s;
            __syncthreads();
            s = l < warps ? slot[at + l] : 0.0f;
            if (l + 16 < warps) s += slot[at + 16 + l];
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        }
        const float t = __shfl_xor_sync(kFull, s, 16);
        return lane & 16 ? make_float2(t, s) : make_float2(s, t);
    }

    template <bool WARP>
    __device__ __forceinline__ float sum(float v)
    {
        v = warp_sum(v);
        if constexpr (!WARP) {
            float *slot = slots[turn];
            turn ^= 1;
            const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
            if (lane == 0) slot[threadIdx.x >> 5] = v;
            __syncthreads();
            v = warp_sum(lane < warps ? slot[lane] : 0.0f);
        }
        return v;
    }

    template <bool WARP>
    __device__ __forceinline__ float max_abs(float m)
    {
        // magnitudes: their bit patterns order like the values
        uint32_t u = __reduce_max_sync(kFull, __float_as_uint(m));
        if constexpr (!WARP) {
            float *slot = slots[turn];
            turn ^= 1;
            const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
            if (lane == 0) slot[threadIdx.x >> 5] = __uint_as_float(u);
            __syncthreads();
            u = __reduce_max_sync(kFull, lane < warps ? __float_as_uint(slot[lane]) : 0u);
        }
        return __uint_as_float(u);
    }
};

// The columns of thread t of a row: vectors t, t + threads, ...; V elements each.
// Loads read the row's first vector in place of one beyond C: without a branch for
// each vector all of a thread's loads are in flight together.
template <int V, int I>
struct Span {
    int t, threads, C;
    __device__ __forceinline__ int col(int i) const { return (t + i * threads) * V; }
    __device__ __forceinline__ bool in(int i) const { return col(i) < C; }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, float *v) const  // anything beyond C
    {
#pragma unroll
        for (int i = 0; i < I; ++i) load_v<V>(row + (in(i) ? col(i) : 0), v + i * V);
    }
    // 0 beyond C
    __device__ __forceinline__ void clear(float *v) const
    {
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) v[i * V + e] = in(i) ? v[i * V + e] : 0.0f;
    }
    // `other` everywhere without a row
    template <typename T>
    __device__ __forceinline__ void load_or(const T *row, float *v, float other) const
    {
        if (row) load(row, v);
        else
#pragma unroll
            for (int e = 0; e < V * I; ++e) v[e] = other;
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, const float *v) const
    {
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (in(i)) store_v<V>(row + col(i), v + i * V);
    }
};

struct Stats {
    float mean, rstd;
};

// sum / C: the product with the rounded 1 / C, put right by its remainder (exact where the
// quotient is a float), so that rows of equal values whose sum is exact are centred to zero at
// every width.  (With a division 12608 x 768 took 35.0 us, not 28.6.)
__device__ __forceinline__ float mean_of(float sum, int C, float inv_c)
{
    const float q = sum * inv_c;
    return __fmaf_rn(__fmaf_rn(-q, (float)C, sum), inv_c, q);
}

// The mean first: as v rstd - mean rstd, one fused operation, the rounding of mean rstd would
// stay where the two terms cancel (up to 0.016 on rows of equal values of 1000, eps 1e-5).
__device__ __forceinline__ float normalised(float v, const Stats &s) { return (v - s.mean) * s.rstd; }

// 1 / sqrt(ss / C + eps) (2 ulp of the fp32 value, beside sums of many roundings)
__device__ __forceinline__ float rstd_of(float ss, float inv_c, float eps) { return rsqrtf(__fmaf_rn(ss, inv_c, eps)); }

// One row's statistics; columns beyond C (zeros in v) are left out of the variance.
template <bool WARP, int V, int I>
__device__ __forceinline__ Stats row_stats(const Span<V, I> &sp, const float *v, int kind, float eps, float inv_c,
                                           RowReduce &red)
{
    Stats s{0.0f, 0.0f};
    float acc = 0.0f;
    if (kind == QNN_NORM_LAYER) {
#pragma unroll
        for (int e = 0; e < V * I; ++e) acc += v[e];
        s.mean = mean_of(red.sum<WARP>(acc), sp.C, inv_c);
        acc = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (sp.in(i))
#pragma unroll
                for (int e = i * V; e < (i + 1) * V; ++e) {
                    const float d = v[e] - s.mean;
                    acc = __fmaf_rn(d, d, acc);
                }
    } else {
#pragma unroll
        for (int e = 0; e < V * I; ++e) acc = __fmaf_rn(v[e], v[e], acc);
    }
    s.rstd = rstd_of(red.sum<WARP>(acc), inv_c, eps);
    return s;
}

// Rows come to shared memory in whole 16-byte pieces: the window around a row, which
// starts `off` bytes into it (V = 8: rows on such boundaries, off = 0).  A window reaches
// up to 15 bytes past its row; rows whose windows could leave the tensor, the last ones,
// are not copied (ring_rows).
template <int V>
__host__ __device__ inline int window_room(int C, int elem)
{
    return V == 8 ? C * elem : (C * elem + 30) & ~15;
}

struct Window {
    const uint8_t *src;
    uint32_t off, bytes;
};

template <int V, typename T>
__device__ __forceinline__ Window window(const void *base, int64_t row, int64_t ld, int C)
{
    const int64_t at = row * ld * (int)sizeof(T);
    const uint32_t off = V == 8 ? 0 : (uint32_t)at & 15u;
    return {static_cast<const uint8_t *>(base) + (at - off), off, (off + (uint32_t)C * (uint32_t)sizeof(T) + 15u) & ~15u};
}

// Leading rows of `rows` whose windows stay inside a tensor of pitch ld.
inline int64_t ring_rows(int64_t rows, int64_t ld, int elem)
{
    const int64_t pitch = std::min<int64_t>(ld, 16) * elem;  // from 15 bytes on, the last row alone
    return std::max<int64_t>(0, rows - (15 + pitch - 1) / pitch);
}

// After a wait that gave up: waits, each with its limit, for the ring's other copies in
// flight, `left` rows from `stage` on at most, so that none writes to memory given back.
__device__ __forceinline__ void drain_ring(uint32_t bar0, int stages, int stage, uint32_t phase, int64_t left,
                                           uint32_t *status)
{
    for (int i = 0; i < stages && i < left; ++i) {
        (void)mbar_wait(bar0 + 8 * stage, phase, status);
        if (++stage == stages) stage = 0, phase ^= 1;
    }
}

// ---- host ----------------------------------------------------------------------------


bool norm_ok(int kind) { return kind == QNN_NORM_NONE || kind == QNN_NORM_RMS || kind == QNN_NORM_LAYER; }
bool is_finite(float v) { return v == v && v < INFINITY && v > -INFINITY; }

// What both directions check of the sizes, types and parameters.
qnn_status check_params(int r_dt, const void *y, int y_dt, int64_t rows, int C, const qnn_block_norm *p)
{
    if (!p || rows < 0 || C <= 0 || !norm_ok(p->post) || !norm_ok(p->pre) || p->gate_rows < 0 || p->ld_r < 0 ||
        p->ld_y < 0 || p->ld_h < 0)
        return QNN_ERR_INVALID_ARG;
    if (!is_finite(p->res_scale) || !is_finite(p->block_scale) || !is_finite(p->eps_post) || !is_finite(p->eps_pre) ||
        p->eps_post < 0 || p->eps_pre < 0)
        return QNN_ERR_INVALID_ARG;
    if ((p->ld_r && p->ld_r < C) || (p->ld_y && p->ld_y < C) || (p->ld_h && p->ld_h < C)) return QNN_ERR_INVALID_ARG;
    if (!is_float_dt(y_dt) || (r_dt != y_dt && r_dt != QNN_F32) || C > kMaxC) return QNN_ERR_UNSUPPORTED;
    if (!y && rows > 0 && (p->post != QNN_NORM_NONE || p->gate)) return QNN_ERR_INVALID_ARG;
    if ((p->post == QNN_NORM_NONE && (p->gamma_post || p->beta_post)) ||
        (p->pre == QNN_NORM_NONE && (p->gamma_pre || p->beta_pre)))
        return QNN_ERR_INVALID_ARG;
    const void *ptr[] = {p->gamma_post, p->beta_post, p->gamma_pre, p->beta_pre, p->gate};
    for (const void *q : ptr)
        if (!aligned16(q)) return QNN_ERR_ALIGNMENT;
    return QNN_OK;
}

bool rows_aligned(int64_t ld, int bytes) { return ld * bytes % 16 == 0; }

// fn(row type, block type) for the pair of types
template <typename F>
void with_types(int r_dt, int y_dt, F fn)
{
    if (y_dt == QNN_F32) fn(float{}, float{});
    else if (y_dt == QNN_F16 && r_dt == QNN_F32) fn(float{}, __half{});
    else if (y_dt == QNN_F16) fn(__half{}, __half{});
    else if (r_dt == QNN_F32) fn(float{}, __nv_bfloat16{});
    else fn(__nv_bfloat16{}, __nv_bfloat16{});
}

// Launch as the programmatic dependent of the grid before on the stream: every thread
// waits for that grid before it touches global memory.
template <typename K, typename A>
qnn_status launch_dependent(K kern, const A &a, dim3 grid, int threads, int smem, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return QNN_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace qnn
