// qnn_blocknorm.cu -- q_block_norm and q_block_norm_backward: the norm after a block,
// its gate and residual scale, the residual add and the norm before the next block,
// row by row in one pass.
//
//   p  = norm_post(y)      r' = a r + b gate p      h = norm_pre(r')
//
// norm: x^ = x / sqrt(mean(x^2) + eps)  (RMS)  or  (x - mean) / sqrt(var + eps)
// (LAYER), then gamma x^ + beta.  Backward, with G the gradient at r':
//   G   = dr' + D_pre(gamma_pre dh),   dr = a G,   t = b gate G,   dy = D_post(gamma_post t)
//   D(g) = (g - mean(g) [LAYER only] - x^ mean(g x^)) / sqrt(...)
//   dgate = b sum G p over the rows that share it;   dgamma = sum upstream x^,
//   dbeta = sum upstream   (upstream: dh before, t after)
//
// Both are bound by the bytes of the rows.  A row is read once and lives in registers
// to its writes: one warp holds rows of up to 1024 columns, a block longer ones.
// Statistics are fp32, the variance from the centred values (a second reduction over
// registers, not over memory).  h is formed from r' before r' is rounded to its own
// type; the backward pass takes its statistics from r' as stored.
//
// Many rows on 16-byte boundaries: the rows to come are on their way to shared memory
// by bulk copies while one is computed (the copies in flight, not registers, are what
// covers the memory's latency).  Few rows, and rows off those boundaries: direct loads.
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
constexpr int kWarpRows = 4;  // warps (rows) per block where a warp holds a row
constexpr int kMaxStages = 4;
// Shared memory of an SM given to rings: what covers the latency twice over; the rest
// stays L1, which holds the parameters.
constexpr int kRingSmem = 128 << 10;

struct NormArgs {
    const void *r, *y, *gate;
    const float *gamma_post, *beta_post, *gamma_pre, *beta_pre;
    void *r_out, *h;
    float *h_scale;
    int64_t rows, ld_r, ld_y, ld_h, gate_rows;
    float a, b, eps_post, eps_pre, inv_c;
    int C, post, pre, s8;
    int small_rows;    // row and gate_rows fit 32 bits
    int stages;        // of a ring
    uint32_t *status;  // device status word
};

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

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float2 warp_sum(float2 v) { return make_float2(warp_sum(v.x), warp_sum(v.y)); }

// Sums (or maxima) over a row's threads: a warp, or the block through shared memory.
// Two slots used in turn make one barrier per call enough: a slot is written again
// only behind the barrier that follows its last read.
struct RowReduce {
    float2 (*slots)[32];
    int turn = 0;

    template <bool WARP>
    __device__ __forceinline__ float2 sum(float2 v)
    {
        v = warp_sum(v);
        if constexpr (!WARP) {
            float2 *s = slots[turn];
            turn ^= 1;
            const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
            if (lane == 0) s[threadIdx.x >> 5] = v;
            __syncthreads();
            v = warp_sum(lane < warps ? s[lane] : make_float2(0.0f, 0.0f));
        }
        return v;
    }

    template <bool WARP>
    __device__ __forceinline__ float sum(float v)
    {
        v = warp_sum(v);
        if constexpr (!WARP) {
            float2 *s = slots[turn];
            turn ^= 1;
            const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
            if (lane == 0) s[threadIdx.x >> 5].x = v;
            __syncthreads();
            v = warp_sum(lane < warps ? s[lane].x : 0.0f);
        }
        return v;
    }

    template <bool WARP>
    __device__ __forceinline__ float max_abs(float m)
    {
        // magnitudes: their bit patterns order like the values
        uint32_t u = __reduce_max_sync(kFull, __float_as_uint(m));
        if constexpr (!WARP) {
            float2 *s = slots[turn];
            turn ^= 1;
            const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
            if (lane == 0) s[threadIdx.x >> 5] = make_float2(__uint_as_float(u), 0.0f);
            __syncthreads();
            u = __reduce_max_sync(kFull, lane < warps ? __float_as_uint(s[lane].x) : 0u);
        }
        return __uint_as_float(u);
    }
};

// rint(t) of |t| <= 128 in the low byte: adding 1.5 2^23 leaves the integer in the low
// bits of the sum, rounded half to even.
__device__ __forceinline__ uint32_t low_int(float t) { return __float_as_uint(t + 12582912.0f); }

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return prmt(prmt(a, b, 0x0040), prmt(c, d, 0x0040), 0x5410);
}

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
    template <typename T>
    __device__ __forceinline__ void load0(const T *row, float *v) const
    {
        load(row, v);
        clear(v);
    }
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

__device__ __forceinline__ float rstd_of(float ss, float inv_c, float eps)
{
    return __frcp_rn(__fsqrt_rn(__fmaf_rn(ss, inv_c, eps)));
}

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
        s.mean = red.sum<WARP>(acc) * inv_c;
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

// v = (v - mean) rstd
template <int V, int I>
__device__ __forceinline__ void normalise(const Span<V, I> &sp, float *v, const Stats &s)
{
#pragma unroll
    for (int i = 0; i < I; ++i)
        if (sp.in(i))
#pragma unroll
            for (int e = i * V; e < (i + 1) * V; ++e) v[e] = (v[e] - s.mean) * s.rstd;
}

// v = gamma (v - mean) rstd + beta, (v - mean) rstd as one fused operation.
template <int V, int I>
__device__ __forceinline__ void affine(const Span<V, I> &sp, float *v, const Stats &s, const float *gamma,
                                       const float *beta)
{
    const float c = -s.mean * s.rstd;
    float p[V * I];
#pragma unroll
    for (int e = 0; e < V * I; ++e) v[e] = __fmaf_rn(v[e], s.rstd, c);
    if (gamma) {
        sp.load(gamma, p);
#pragma unroll
        for (int e = 0; e < V * I; ++e) v[e] *= p[e];
    }
    if (beta) {
        sp.load(beta, p);
#pragma unroll
        for (int e = 0; e < V * I; ++e) v[e] += p[e];
    }
}

// One row from its pointers (y and g may be null).  EARLY: all loads before the first
// reduction (few rows: one wait for memory, not three).  release() is called once the
// row has been read by all its threads, unless EARLY.
template <typename TR, typename TY, bool WARP, bool EARLY, int V, int I, typename F>
__device__ __forceinline__ void norm_row(const NormArgs &a, const Span<V, I> &sp, int64_t row, const TR *r,
                                         const TY *y, const TY *g, RowReduce &red, F release)
{
    constexpr int E = V * I, L = EARLY ? E : 1;
    float v[E], t[E], ge[L], gm[L], bt[L], hm[L], hb[L];
    sp.load_or(y, v, 0.0f);
    if constexpr (EARLY) {
        sp.load(r, t);
        sp.load_or(g, ge, 1.0f);
        sp.load_or(a.gamma_post, gm, 1.0f);
        sp.load_or(a.beta_post, bt, 0.0f);
        sp.load_or(a.gamma_pre, hm, 1.0f);
        sp.load_or(a.beta_pre, hb, 0.0f);
    }
    if (a.post != QNN_NORM_NONE) {
        sp.clear(v);
        const Stats s = row_stats<WARP>(sp, v, a.post, a.eps_post, a.inv_c, red);
        if constexpr (EARLY) {
            const float c = -s.mean * s.rstd;
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __fmaf_rn(__fmaf_rn(v[e], s.rstd, c), gm[e], bt[e]);
        } else {
            affine(sp, v, s, a.gamma_post, a.beta_post);
        }
    }
    if constexpr (EARLY) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= ge[e];
    } else {
        if (g) {
            sp.load(g, t);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= t[e];
        }
        sp.load(r, t);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __fmaf_rn(a.b, v[e], a.a * t[e]);
    if (a.r_out) sp.store(static_cast<TR *>(a.r_out) + row * a.ld_r, v);
    if (!EARLY && (WARP || a.pre == QNN_NORM_NONE)) {
        if constexpr (WARP) __syncwarp();
        else __syncthreads();
        release();
    }
    if (!a.h) return;
    sp.clear(v);
    if (a.pre != QNN_NORM_NONE) {
        const Stats s = row_stats<WARP>(sp, v, a.pre, a.eps_pre, a.inv_c, red);
        if (!EARLY && !WARP) release();
        if constexpr (EARLY) {
            const float c = -s.mean * s.rstd;
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __fmaf_rn(__fmaf_rn(v[e], s.rstd, c), hm[e], hb[e]);
        } else {
            affine(sp, v, s, a.gamma_pre, a.beta_pre);
        }
    }
    if (!a.s8) {
        sp.store(static_cast<TY *>(a.h) + row * a.ld_h, v);
        return;
    }
    float m = 0.0f;
    sp.clear(v);
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(v[e]));
    m = red.max_abs<WARP>(m);
    const float f = m == 0.0f ? 0.0f : __fdiv_rn(127.0f, m);
    if (sp.t == 0) a.h_scale[row] = __fdiv_rn(m, 127.0f);
    int8_t *hr = static_cast<int8_t *>(a.h) + row * a.ld_h;
#pragma unroll
    for (int i = 0; i < I; ++i)
        if (sp.in(i)) {
            if constexpr (V == 1) {
                hr[sp.col(i)] = (int8_t)low_int(v[i] * f);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = low_int(v[i * V + e] * f);
                *reinterpret_cast<uint2 *>(hr + sp.col(i)) =
                    make_uint2(pack4(w[0], w[1], w[2], w[3]), pack4(w[4], w[5], w[6], w[7]));
            }
        }
}

template <typename TY>
__device__ __forceinline__ const TY *gate_row(const NormArgs &a, int64_t row)
{
    if (!a.gate) return nullptr;
    const int64_t q = a.gate_rows == 0 ? 0 : a.gate_rows == 1 ? row : a.small_rows
                          ? (int64_t)((uint32_t)row / (uint32_t)a.gate_rows) : row / a.gate_rows;
    return static_cast<const TY *>(a.gate) + q * a.C;
}

// Rows by direct loads.  MAXT: threads at most.
template <typename TR, typename TY, int V, int I, bool WARP, bool EARLY, int MAXT>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : MAXT)
    block_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float2 slots[2][32];
    RowReduce red{slots};
    const Span<V, I> sp{(int)(WARP ? threadIdx.x & 31 : threadIdx.x), (int)(WARP ? 32 : blockDim.x), a.C};
    const int64_t first = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
    grid_dependency_launch();
    grid_dependency_wait();
    for (int64_t row = first; row < a.rows; row += step) {
        norm_row<TR, TY, WARP, EARLY>(a, sp, row, static_cast<const TR *>(a.r) + row * a.ld_r,
                                      a.y ? static_cast<const TY *>(a.y) + row * a.ld_y : nullptr, gate_row<TY>(a, row),
                                      red, [] {});
    }
}

// Rows through a ring of `stages` in shared memory, each [r][y][gate row, when every
// row has its own]; a warp (WARP) or a block to a ring.  A stage is asked for again
// behind the reduction that follows its last reads.
template <typename TR, typename TY, int I, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 256)
    block_norm_ring_kernel(const __grid_constant__ NormArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 slots[2][32];
    __shared__ __align__(8) uint64_t bars[WARP ? kWarpRows : 1][kMaxStages];
    RowReduce red{slots};
    const int w = WARP ? threadIdx.x >> 5 : 0;
    const Span<8, I> sp{(int)(WARP ? threadIdx.x & 31 : threadIdx.x), (int)(WARP ? 32 : blockDim.x), a.C};
    const int64_t first = WARP ? (int64_t)blockIdx.x * kWarpRows + w : blockIdx.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
    const int rb = a.C * (int)sizeof(TR), yb = a.y ? a.C * (int)sizeof(TY) : 0,
              gb = a.gate && a.gate_rows == 1 ? a.C * (int)sizeof(TY) : 0, bytes = rb + yb + gb;
    uint8_t *ring = smem + (size_t)w * a.stages * bytes;
    const uint32_t bar0 = smem_u32(&bars[w][0]);
    auto ask = [&](int64_t row, int stage) {  // by one thread
        const uint32_t bar = bar0 + 8 * stage, to = smem_u32(ring + (size_t)stage * bytes);
        mbar_arrive_expect_tx(bar, bytes);
        bulk_g2s(to, static_cast<const TR *>(a.r) + row * a.ld_r, rb, bar);
        if (yb) bulk_g2s(to + rb, static_cast<const TY *>(a.y) + row * a.ld_y, yb, bar);
        if (gb) bulk_g2s(to + rb + yb, static_cast<const TY *>(a.gate) + row * a.C, gb, bar);
    };
    grid_dependency_launch();
    if (sp.t == 0) {
        for (int i = 0; i < a.stages; ++i) mbar_init(bar0 + 8 * i, 1);
        fence_mbar_init();
        grid_dependency_wait();
        for (int i = 0; i < a.stages && first + i * step < a.rows; ++i) ask(first + i * step, i);
    }
    if constexpr (WARP) __syncwarp();
    else __syncthreads();
    grid_dependency_wait();
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t row = first; row < a.rows; row += step) {
        if (!mbar_wait(bar0 + 8 * stage, phase, a.status)) return;
        const uint8_t *from = ring + (size_t)stage * bytes;
        norm_row<TR, TY, WARP, false>(
            a, sp, row, reinterpret_cast<const TR *>(from), yb ? reinterpret_cast<const TY *>(from + rb) : nullptr,
            gb ? reinterpret_cast<const TY *>(from + rb + yb) : gate_row<TY>(a, row), red, [&] {
                if (sp.t == 0 && row + a.stages * step < a.rows) ask(row + a.stages * step, stage);
            });
        if (++stage == a.stages) stage = 0, phase ^= 1;
    }
}

// ---- backward ------------------------------------------------------------------------

struct BackArgs {
    const void *r, *y, *gate, *dh, *dr_out;  // r: r' as the forward call wrote it
    const float *gamma_post, *beta_post, *gamma_pre;
    void *dr, *dy, *dgate;
    float *ws;       // [block][kSlots][C]
    uint32_t wants;  // bit s: slot s is summed
    int64_t rows, ld_r, ld_y, ld_h, gate_rows, chunk;
    float a, b, eps_post, eps_pre, inv_c;
    int C, post, pre;
};

// A block's partial sums: the four parameter gradients, and the gate's gradient for a
// group of rows that began in an earlier block's chunk, or that goes on in a later one's.
enum { kGammaPre, kBetaPre, kGammaPost, kBetaPost, kGateHead, kGateTail, kSlots };

template <typename TR, typename TY, int V, int I>
__global__ void __launch_bounds__(1024) block_norm_backward_kernel(const __grid_constant__ BackArgs a)
{
    __shared__ float2 slots[2][32];
    RowReduce red{slots};
    const Span<V, I> sp{(int)threadIdx.x, (int)blockDim.x, a.C};
    const int64_t row0 = blockIdx.x * a.chunk, row1 = min(row0 + a.chunk, a.rows);
    float *part = a.ws + (int64_t)blockIdx.x * kSlots * a.C;
    float gsum[V * I] = {};  // the gate's gradient over the rows of the current group
    auto add = [&](int slot, bool fresh, const float *v) {  // each thread its own columns
        if (!(a.wants >> slot & 1)) return;
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (sp.in(i)) {
                float *p = part + (int64_t)slot * a.C + sp.col(i);
                float o[V];
                if (!fresh) load_v<V>(p, o);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = fresh ? v[i * V + e] : o[e] + v[i * V + e];
                store_v<V>(p, o);
            }
    };
    for (int64_t row = row0; row < row1; ++row) {
        const bool fresh = row == row0;
        float G[V * I], x[V * I], d[V * I];
        if (a.dr_out) sp.load0(static_cast<const TR *>(a.dr_out) + row * a.ld_r, G);
        else
#pragma unroll
            for (int e = 0; e < V * I; ++e) G[e] = 0.0f;
        if (a.dh) {
            sp.load0(static_cast<const TY *>(a.dh) + row * a.ld_h, d);
            if (a.pre != QNN_NORM_NONE) {
                sp.load0(static_cast<const TR *>(a.r) + row * a.ld_r, x);
                const Stats s = row_stats<false>(sp, x, a.pre, a.eps_pre, a.inv_c, red);
                normalise(sp, x, s);
                add(kBetaPre, fresh, d);
                float t[V * I];
                float2 m = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    float gm[V];
                    if (sp.in(i) && a.gamma_pre) load_v<V>(a.gamma_pre + sp.col(i), gm);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int k = i * V + e;
                        t[k] = d[k] * x[k];
                        if (sp.in(i) && a.gamma_pre) d[k] *= gm[e];
                        m.x += d[k];
                        m.y = __fmaf_rn(d[k], x[k], m.y);
                    }
                }
                add(kGammaPre, fresh, t);
                m = red.sum<false>(m);
                const float mg = a.pre == QNN_NORM_LAYER ? m.x * a.inv_c : 0.0f, mx = m.y * a.inv_c;
#pragma unroll
                for (int i = 0; i < I; ++i)
                    if (sp.in(i))  // columns beyond C stay zero, in the sums to come too
#pragma unroll
                        for (int e = i * V; e < (i + 1) * V; ++e)
                            G[e] = __fmaf_rn(s.rstd, __fmaf_rn(-x[e], mx, d[e] - mg), G[e]);
            } else {
#pragma unroll
                for (int e = 0; e < V * I; ++e) G[e] += d[e];
            }
        }
        if (a.dr) {
#pragma unroll
            for (int e = 0; e < V * I; ++e) d[e] = a.a * G[e];
            sp.store(static_cast<TR *>(a.dr) + row * a.ld_r, d);
        }
        if (!a.y) continue;
        // x = y^ (or y), d = t = b gate G, gsum += b G p
        sp.load0(static_cast<const TY *>(a.y) + row * a.ld_y, x);
        Stats s{0.0f, 1.0f};
        if (a.post != QNN_NORM_NONE) {
            s = row_stats<false>(sp, x, a.post, a.eps_post, a.inv_c, red);
            normalise(sp, x, s);
        }
        const int64_t q = a.gate_rows ? row / a.gate_rows : 0;
        float2 m = make_float2(0.0f, 0.0f);
        float t[V * I];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float gm[V], bt[V], gt[V];
            if (sp.in(i)) {
                if (a.gamma_post) load_v<V>(a.gamma_post + sp.col(i), gm);
                if (a.beta_post) load_v<V>(a.beta_post + sp.col(i), bt);
                if (a.gate) load_v<V>(static_cast<const TY *>(a.gate) + q * a.C + sp.col(i), gt);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int k = i * V + e;
                float p = x[k];
                d[k] = a.b * G[k];
                if (sp.in(i)) {
                    if (a.gamma_post) p *= gm[e];
                    if (a.beta_post) p += bt[e];
                    gsum[k] = __fmaf_rn(d[k], p, gsum[k]);
                    if (a.gate) d[k] *= gt[e];
                }
                t[k] = d[k] * x[k];
            }
        }
        add(kBetaPost, fresh, d);
        add(kGammaPost, fresh, t);
        if (a.dy) {
            if (a.post != QNN_NORM_NONE) {
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    float gm[V];
                    if (sp.in(i) && a.gamma_post) load_v<V>(a.gamma_post + sp.col(i), gm);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int k = i * V + e;
                        if (sp.in(i) && a.gamma_post) d[k] *= gm[e];
                        m.x += d[k];
                        m.y = __fmaf_rn(d[k], x[k], m.y);
                    }
                }
                m = red.sum<false>(m);
                const float mg = a.post == QNN_NORM_LAYER ? m.x * a.inv_c : 0.0f, mx = m.y * a.inv_c;
#pragma unroll
                for (int e = 0; e < V * I; ++e) d[e] = s.rstd * __fmaf_rn(-x[e], mx, d[e] - mg);
            }
            sp.store(static_cast<TY *>(a.dy) + row * a.ld_y, d);
        }
        if (!a.dgate) continue;
        // the group ends with this row, or the chunk does
        const int64_t end = a.gate_rows ? min((q + 1) * a.gate_rows, a.rows) : a.rows;
        if (row + 1 == end || row + 1 == row1) {
            const bool began = q * a.gate_rows >= row0;
            if (began && row + 1 == end) sp.store(static_cast<TY *>(a.dgate) + q * a.C, gsum);
            else add(began ? kGateTail : kGateHead, true, gsum);
#pragma unroll
            for (int e = 0; e < V * I; ++e) gsum[e] = 0.0f;
        }
    }
}

struct FinishArgs {
    const float *ws;
    float *out[4];  // dgamma_pre, dbeta_pre, dgamma_post, dbeta_post
    void *dgate;
    int64_t rows, gate_rows, chunk;
    int C, blocks, gate_dt;
};

// Adds the blocks' partial sums in a fixed order.  blockIdx.y: one of the four parameter
// gradients, then the boundaries between two blocks' rows, for the group of rows that
// shares a gate across it (a group across several is done at its first).  32 columns a
// block, its 8 warps taking every eighth partial.
__global__ void __launch_bounds__(256) block_norm_finish_kernel(const __grid_constant__ FinishArgs a)
{
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane, job = blockIdx.y;
    int b0 = 0, b1 = a.blocks;
    int64_t q = 0;
    if (job < 4) {
        if (!a.out[job]) return;
    } else {
        const int b = job - 3;  // the boundary before block b
        q = a.gate_rows ? b * a.chunk / a.gate_rows : 0;
        const int64_t r0 = q * a.gate_rows, r1 = a.gate_rows ? min(r0 + a.gate_rows, a.rows) : a.rows;
        if (r0 == b * a.chunk || r0 / a.chunk != b - 1) return;
        b0 = b - 1;
        b1 = (int)((r1 - 1) / a.chunk) + 1;
    }
    float v = 0.0f;
    if (col < a.C)
        for (int b = b0 + w; b < b1; b += 8) {
            const int slot = job < 4 ? job : b == b0 ? kGateTail : kGateHead;
            v += a.ws[((int64_t)b * kSlots + slot) * a.C + col];
        }
    s[w][lane] = v;
    __syncthreads();
    if (w != 0 || col >= a.C) return;
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += s[k][lane];
    const int64_t at = q * a.C + col;
    if (job < 4) a.out[job][col] = v;
    else if (a.gate_dt == QNN_F32) static_cast<float *>(a.dgate)[at] = v;
    else if (a.gate_dt == QNN_F16) static_cast<__half *>(a.dgate)[at] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16 *>(a.dgate)[at] = from_f32<__nv_bfloat16>(v);
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
qnn_status launch_dependent(K kern, const A &a, int64_t grid, int threads, int smem, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
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

template <typename TR, typename TY, int V, int I, int MAXT>
qnn_status launch_norm(const NormArgs &a, cudaStream_t s)
{
    constexpr int per = V * I;
    if (a.C <= 32 * per && MAXT <= 512)
        return launch_dependent(block_norm_kernel<TR, TY, V, I, true, per <= 8, 512>, a,
                                std::min<int64_t>((a.rows + kWarpRows - 1) / kWarpRows, 16 * sm_count()),
                                32 * kWarpRows, 0, s);
    const int threads = (a.C + per * 32 - 1) / (per * 32) * 32;
    return launch_dependent(block_norm_kernel<TR, TY, V, I, false, per <= 8, MAXT>, a,
                            std::min<int64_t>(a.rows, (int64_t)sm_count() * std::max(1024 / threads, 1)), threads, 0, s);
}

template <typename TR, typename TY, int I, bool WARP>
qnn_status launch_ring(NormArgs a, cudaStream_t s)
{
    const int rows = WARP ? kWarpRows : 1, threads = WARP ? 32 * kWarpRows : (a.C + I * 256 - 1) / (I * 256) * 32;
    const int stage = rows * a.C * (int)(sizeof(TR) + (a.y ? sizeof(TY) : 0) +
                                         (a.gate && a.gate_rows == 1 ? sizeof(TY) : 0));
    // as many blocks on an SM as its registers hold, their rings in what there is for them
    constexpr int most = I == 1 ? 1280 : I == 2 ? 1024 : I == 3 ? 768 : 640;  // threads
    const int blocks = std::max(1, std::min(kRingSmem / stage, most / threads));
    a.stages = std::max(1, std::min(kMaxStages, kRingSmem / (blocks * stage)));
    auto kern = block_norm_ring_kernel<TR, TY, I, WARP>;
    static std::atomic<uint64_t> opted_in{0};
    if (!opt_in_smem(kern, kRingSmem, opted_in, 60)) return QNN_ERR_CUDA;
    const int64_t want = (a.rows + rows - 1) / rows;
    return launch_dependent(kern, a, std::min<int64_t>(want, (int64_t)sm_count() * blocks), threads, a.stages * stage, s);
}

// Rows per block of the backward pass: two blocks' worth of rows for each SM, and no
// fewer than 8 rows a block, so that the partial sums stay small beside the rows.
int64_t back_chunk(int64_t rows) { return std::max<int64_t>((rows + 2 * sm_count() - 1) / (2 * sm_count()), 8); }
int64_t back_blocks(int64_t rows) { return rows ? (rows + back_chunk(rows) - 1) / back_chunk(rows) : 0; }

template <typename TR, typename TY, int V, int I>
void launch_back(const BackArgs &a, cudaStream_t s)
{
    const int per = V * I * 32;
    block_norm_backward_kernel<TR, TY, V, I>
        <<<(int)back_blocks(a.rows), (a.C + per - 1) / per * 32, 0, s>>>(a);
}

}  // namespace
}  // namespace qnn

extern "C" qnn_status q_block_norm(const void *r, qnn_dtype r_dt, const void *y, qnn_dtype y_dt, int64_t rows, int C,
                                   const qnn_block_norm *p, void *r_out, void *h, qnn_dtype h_dt, float *h_scale,
                                   qnn_stream_t stream)
{
    using namespace qnn;
    const qnn_status st = check_params(r_dt, y, y_dt, rows, C, p);
    if (st != QNN_OK) return st;
    const bool s8 = h_dt == QNN_S8;
    if (!s8 && h_dt != y_dt) return QNN_ERR_UNSUPPORTED;
    if (rows == 0) return QNN_OK;
    if (!r || (!r_out && !h) || (h && s8) != (h_scale != nullptr)) return QNN_ERR_INVALID_ARG;
    if (!aligned16(r) || !aligned16(y) || !aligned16(r_out) || !aligned16(h) || !aligned16(h_scale))
        return QNN_ERR_ALIGNMENT;
    NormArgs a{};
    a.r = r, a.y = y, a.gate = p->gate, a.r_out = r_out, a.h = h, a.h_scale = h_scale;
    a.gamma_post = p->gamma_post, a.beta_post = p->beta_post, a.gamma_pre = p->gamma_pre, a.beta_pre = p->beta_pre;
    a.rows = rows, a.gate_rows = p->gate_rows, a.C = C, a.post = p->post, a.pre = p->pre, a.s8 = s8;
    a.ld_r = p->ld_r ? p->ld_r : C, a.ld_y = p->ld_y ? p->ld_y : C, a.ld_h = p->ld_h ? p->ld_h : C;
    a.a = p->res_scale, a.b = p->block_scale, a.eps_post = p->eps_post, a.eps_pre = p->eps_pre, a.inv_c = 1.0f / C;
    const int ey = float_bytes(y_dt);
    const bool vec = C % 8 == 0 && rows_aligned(a.ld_r, float_bytes(r_dt)) && (!y || rows_aligned(a.ld_y, ey)) &&
                     (!h || (s8 ? a.ld_h % 8 == 0 : rows_aligned(a.ld_h, ey)));
    a.small_rows = rows <= INT32_MAX && p->gate_rows <= INT32_MAX;
    a.status = status_word();
    if (!a.status) return QNN_ERR_CUDA;
    // rings from the size on at which every SM has several rows to go through
    const int row_bytes = C * (float_bytes(r_dt) + (y ? ey : 0) + (p->gate && p->gate_rows == 1 ? ey : 0));
    const bool many = rows * C >= (int64_t)sm_count() * 16384, ring = many && vec && C <= 8192 && row_bytes <= kRingSmem;
    cudaStream_t s = (cudaStream_t)stream;
    qnn_status done = QNN_OK;
    with_types(r_dt, y_dt, [&](auto tr, auto ty) {
        using TR = decltype(tr);
        using TY = decltype(ty);
        if (ring && C <= 256) done = launch_ring<TR, TY, 1, true>(a, s);
        else if (ring && C <= 512) done = launch_ring<TR, TY, 2, true>(a, s);
        else if (ring && C <= 768) done = launch_ring<TR, TY, 3, true>(a, s);
        else if (ring && C <= 1024) done = launch_ring<TR, TY, 4, true>(a, s);
        else if (ring) done = launch_ring<TR, TY, 4, false>(a, s);
        else if (vec && C <= 4096) done = launch_norm<TR, TY, 8, 1, 512>(a, s);
        else if (vec) done = launch_norm<TR, TY, 8, 4, 1024>(a, s);
        else if (C <= 4096 && !many) done = launch_norm<TR, TY, 1, 8, 512>(a, s);
        else if (C <= 4096) done = launch_norm<TR, TY, 1, 16, 512>(a, s);
        else done = launch_norm<TR, TY, 1, 32, 1024>(a, s);
    });
    return done;
}

extern "C" size_t qnn_block_norm_backward_workspace_bytes(int64_t rows, int C, const qnn_block_norm *p)
{
    if (!p || rows < 0 || C <= 0 || C > qnn::kMaxC) return 0;
    return (size_t)qnn::back_blocks(rows) * qnn::kSlots * C * sizeof(float);
}

extern "C" qnn_status q_block_norm_backward(const void *r_out, qnn_dtype r_dt, const void *y, qnn_dtype y_dt,
                                            int64_t rows, int C, const qnn_block_norm *p, const void *dh,
                                            const void *dr_out, void *dr, void *dy, void *dgate, float *dgamma_pre,
                                            float *dbeta_pre, float *dgamma_post, float *dbeta_post, void *workspace,
                                            size_t workspace_bytes, qnn_stream_t stream)
{
    using namespace qnn;
    const qnn_status st = check_params(r_dt, y, y_dt, rows, C, p);
    if (st != QNN_OK) return st;
    if ((dgate && !p->gate) || (dgamma_pre && !p->gamma_pre) || (dbeta_pre && !p->beta_pre) ||
        (dgamma_post && !p->gamma_post) || (dbeta_post && !p->beta_post))
        return QNN_ERR_INVALID_ARG;
    if (rows > 0) {
        if ((!dh && !dr_out) || (!dh && (dgamma_pre || dbeta_pre)) || (dy && !y)) return QNN_ERR_INVALID_ARG;
        if (dh && p->pre != QNN_NORM_NONE && !r_out) return QNN_ERR_INVALID_ARG;
    }
    const void *ptr[] = {r_out, y, dh, dr_out, dr, dy, dgate, dgamma_pre, dbeta_pre, dgamma_post, dbeta_post,
                         workspace};
    for (const void *q : ptr)
        if (!aligned16(q)) return QNN_ERR_ALIGNMENT;
    const bool sums = dgate || dgamma_pre || dbeta_pre || dgamma_post || dbeta_post;
    if (!sums && !dr && !dy) return QNN_ERR_INVALID_ARG;
    if (sums && rows > 0 && (!workspace || workspace_bytes < qnn_block_norm_backward_workspace_bytes(rows, C, p)))
        return QNN_ERR_INVALID_ARG;
    BackArgs a{};
    a.r = r_out, a.y = y, a.gate = p->gate, a.dh = dh, a.dr_out = dr_out, a.dr = dr, a.dy = dy, a.dgate = dgate;
    a.gamma_post = p->gamma_post, a.beta_post = p->beta_post, a.gamma_pre = p->gamma_pre;
    a.ws = static_cast<float *>(workspace);
    a.rows = rows, a.gate_rows = p->gate_rows, a.C = C, a.post = p->post, a.pre = p->pre, a.chunk = back_chunk(rows);
    a.ld_r = p->ld_r ? p->ld_r : C, a.ld_y = p->ld_y ? p->ld_y : C, a.ld_h = p->ld_h ? p->ld_h : C;
    a.a = p->res_scale, a.b = p->block_scale, a.eps_post = p->eps_post, a.eps_pre = p->eps_pre, a.inv_c = 1.0f / C;
    a.wants = (dgamma_pre ? 1u << kGammaPre : 0) | (dbeta_pre ? 1u << kBetaPre : 0) |
              (dgamma_post ? 1u << kGammaPost : 0) | (dbeta_post ? 1u << kBetaPost : 0) |
              (dgate ? 1u << kGateHead | 1u << kGateTail : 0);
    cudaStream_t s = (cudaStream_t)stream;
    if (rows > 0) {
        const int ey = float_bytes(y_dt);
        const bool vec = C % 8 == 0 && rows_aligned(a.ld_r, float_bytes(r_dt)) && (!y || rows_aligned(a.ld_y, ey)) &&
                         (!dh || rows_aligned(a.ld_h, ey));
        with_types(r_dt, y_dt, [&](auto tr, auto ty) {
            using TR = decltype(tr);
            using TY = decltype(ty);
            if (vec && C <= 8192) launch_back<TR, TY, 8, 1>(a, s);
            else if (vec) launch_back<TR, TY, 8, 4>(a, s);
            else if (C <= 8192) launch_back<TR, TY, 1, 8>(a, s);
            else launch_back<TR, TY, 1, 32>(a, s);
        });
        const qnn_status done = launch_status();
        if (done != QNN_OK || !sums) return done;
    }
    if (!sums) return QNN_OK;
    if (rows == 0 && dgate && !p->gate_rows &&
        cudaMemsetAsync(dgate, 0, (size_t)C * float_bytes(y_dt), s) != cudaSuccess)
        return QNN_ERR_CUDA;
    FinishArgs f{};
    f.ws = a.ws;
    f.out[0] = dgamma_pre, f.out[1] = dbeta_pre, f.out[2] = dgamma_post, f.out[3] = dbeta_post;
    f.dgate = dgate, f.gate_dt = y_dt, f.rows = rows, f.gate_rows = p->gate_rows, f.chunk = a.chunk, f.C = C;
    f.blocks = (int)back_blocks(rows);
    const dim3 grid((C + 31) / 32, dgate ? 4 + std::max(f.blocks - 1, 0) : 4);
    block_norm_finish_kernel<<<grid, 256, 0, s>>>(f);
    return launch_status();
}
