// qnn_gemv.cu -- qgemv_w4: a few rows of activations times 4-bit weights with
// group scales (the weight-only linear layer at decoding sizes).
//
//   y[m][n] = bias[n] + sum_g s[n][g] sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weights are read once and are nearly all the bytes, so the op is bound by the
// weight stream: 23 bytes, 47 codes, a clock and SM.  The SM's integer pipe does 64
// operations a clock, which is not much more, so what is done to a code decides.  The
// codes become f16 integers two at a time (5 integer and 4 f16 operations for 8
// codes, below) and the products run on the tensor cores (mma.sync m16n8k16: 16
// output channels x 8 columns of x).  Converting to bf16 takes 7 integer operations
// for 8 codes, and multiplying on the CUDA cores more than one for each.
//
// x therefore enters as f16, whatever its type: f16 as it is; bf16 and fp32 times a
// power of two for each row (and block) that takes the row's largest finite value
// below 2^14, undone on the sums.  bf16 fits f16's 11 bits; fp32 is the sum of two
// f16, two columns of the operand, to 2^-24 of itself.  Values below 2^-28 of the row's
// largest are held to 2^-39 of that, far under the fp32 rounding of its sums.
//
// The image (prepack): per tile of 16 output channels and step of 128 input
// channels, 1024 bytes, 32 a lane.  A 32-bit word of lane (g, j) (g = lane / 4, j =
// lane % 4) holds channels n = g and g + 8 at four consecutive k: nibbles at bits
// 0/16: (g; k, k+1), 4/20: (g+8; k, k+1), 8/24: (g; k+2, k+3), 12/28: (g+8; k+2, k+3),
// the four registers of the MMA's A fragment.  Word w of the lane covers k =
// 32 (w / 2) + 8 j + 4 (w % 2): the order of K is free, and so a lane's 8 values of x
// for two MMAs are contiguous.  Behind the codes: the scales [tile][group][8][2]
// (channels n, n + 8), then (U4) the zero points in the same order, bytes.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>
#include "qnn_float.cuh"
#include "qnn_internal.h"
#include "qnn_ptx.cuh"

namespace qnn {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;

// one buffer of the warps' sums: [runs][channels of a block][columns, padded]
template <int NT, int R>
constexpr int kPartBytes = kWarps * 16 * R * (NT * 8 + 1) * 4;


struct W4Image {
    int64_t tiles, steps, groups;  // ceil(N / 16), ceil(K / 128), ceil(K / group)
    size_t scale_off, zero_off, total;
};

bool w4_image(const qnn_w4_geom *g, W4Image *im)
{
    if (!g || g->N <= 0 || g->K <= 0 || g->K > (1 << 30) || g->K % 2 != 0 || g->group <= 0 || g->group % 32 != 0) return false;
    if ((g->w_dt != QNN_S4 && g->w_dt != QNN_U4) || !is_float_dt(g->scale_dt)) return false;
    im->tiles = ((int64_t)g->N + 15) / 16;
    im->steps = ((int64_t)g->K + 127) / 128;
    im->groups = ((int64_t)g->K + g->group - 1) / g->group;
    im->scale_off = (size_t)im->tiles * im->steps * 1024;
    im->zero_off = im->scale_off + (size_t)im->tiles * im->groups * 16 * float_bytes(g->scale_dt);
    im->total = im->zero_off + (g->w_dt == QNN_U4 ? (size_t)im->tiles * im->groups * 16 : 0);
    return true;
}

bool aligned_image(const void *p) { return reinterpret_cast<uintptr_t>(p) % 128 == 0; }

// ---- prepack -----------------------------------------------------------------------

// One thread per word of the image; codes outside [N, K) are 0.
// Codes are stored offset: q + 8 for S4, so that both types are u4 with a zero point.
__global__ void __launch_bounds__(256) prepack_w4_kernel(const uint8_t *__restrict__ W, int64_t N, int64_t K,
                                                         int64_t steps, int64_t words, int is_signed,
                                                         uint32_t *__restrict__ out)
{
    const int64_t pitch = K / 2;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int w = (int)(i & 7), lane = (int)(i >> 3) & 31;
        const int64_t step = (i >> 8) % steps, tile = (i >> 8) / steps;
        const int64_t k = step * 128 + (w >> 1) * 32 + (lane & 3) * 8 + (w & 1) * 4;
        uint32_t v = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = tile * 16 + (lane >> 2) + 8 * h;
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // the pair k + 2 e, k + 2 e + 1: one byte
                uint32_t b = 0;
                if (n < N && k + 2 * e < K) b = W[n * pitch + (k >> 1) + e];
                if (is_signed) b ^= 0x88u;
                v |= ((b & 15u) | (b >> 4 << 16)) << (4 * h + 8 * e);
            }
        }
        out[i] = v;
    }
}

// scales (copied bit for bit) and zero points, [N, G] -> [tile][group][8][2]: a lane's two
// channels, n and n + 8, side by side
template <typename T>
__global__ void __launch_bounds__(256) prepack_w4_scale_kernel(const T *__restrict__ scale,
                                                               const int32_t *__restrict__ zero, int64_t N,
                                                               int64_t G, int64_t total, T *__restrict__ out,
                                                               uint8_t *__restrict__ zout, uint32_t *status)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t n = (i >> 4) / G * 16 + (i >> 1 & 7) + 8 * (i & 1), g = (i >> 4) % G;
        out[i] = n < N ? scale[n * G + g] : T(0);
        if (zero) {
            const int32_t z = n < N ? zero[n * G + g] : 0;
            if (z < 0 || z > 15) atomicOr(status, kStatusBadArg);
            zout[i] = (uint8_t)(z & 15);
        }
    }
}

// ---- the product -------------------------------------------------------------------

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
    int vec;         // rows of x start on 16-byte boundaries
    int pass_steps;  // steps of x held in shared memory at a time
    int lane_bits;   // log2 of the threads that share a row of x when it is read
    int sets;        // of ROWS channels
};

// d += a b, a 16 x 16 tile of codes times 16 x 8 of x
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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

// Eight values of x (a "piece") as the 16-bit operand, one or three columns of it.
template <int XT>
__device__ __forceinline__ void put_piece(uint4 u, uint4 w, uint4 *out)
{
    if constexpr (XT != QNN_F32) {
        *out = u;
    } else {
        const uint32_t v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
        uint32_t o[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t lo[3], hi[3];
            bf16_parts(__uint_as_float(v[2 * e]), lo);
            bf16_parts(__uint_as_float(v[2 * e + 1]), hi);
#pragma unroll
            for (int q = 0; q < 3; ++q) o[q][e] = lo[q] | hi[q] << 16;
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) out[4 * q] = make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
    }
}

// Pieces i0 + lane, i0 + lane + share .. < i1 of row `row` of x (at k = k0 + 8 i) to shared
// memory as B fragments, [32 channels][column][j]; zero beyond K.
template <int XT>
__device__ __forceinline__ void stage_x(const GemvArgs &a, int64_t row, int col, int cols, int k0, int i0, int i1,
                                        int lane, int share, uint4 *xs)
{
    constexpr int W = XT == QNN_F32 ? 2 : 1;  // 16-byte words of a piece
    const uint8_t *p = static_cast<const uint8_t *>(a.x) + (row * a.ldx + k0) * (8 * W / 4);
    const int end = a.K - k0, whole = a.vec ? min(i1, end >> 3) : i0;
#pragma unroll 4
    for (int i = i0 + lane; i < whole; i += share) {
        const uint4 *v = reinterpret_cast<const uint4 *>(p) + (int64_t)i * W;
        const uint4 u = __ldg(v);
        put_piece<XT>(u, W == 2 ? __ldg(v + W - 1) : u, xs + ((i >> 2) * cols + col) * 4 + (i & 3));
    }
    // rows off 16-byte boundaries and the ragged end: value by value
#pragma unroll 8
    for (int e = max(whole, i0) * 8 + lane; e < i1 * 8; e += share) {
        uint16_t *out = reinterpret_cast<uint16_t *>(xs + ((e >> 5) * cols + col) * 4 + (e >> 3 & 3)) + (e & 7);
        if constexpr (W == 2) {
            uint32_t v[3];
            bf16_parts(e < end ? __ldg(reinterpret_cast<const float *>(p) + e) : 0.0f, v);
#pragma unroll
            for (int q = 0; q < 3; ++q) out[32 * q] = (uint16_t)v[q];
        } else {
            *out = e < end ? __ldg(reinterpret_cast<const uint16_t *>(p) + e) : (uint16_t)0;
        }
    }
}

// A lane's two scales as they are kept: fp32 in both words, 16-bit types in the first.
__device__ __forceinline__ uint2 load_scales(const uint8_t *p, int dt)
{
    return dt == QNN_F32 ? __ldg(reinterpret_cast<const uint2 *>(p))
                         : make_uint2(__ldg(reinterpret_cast<const uint32_t *>(p)), 0u);
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

// What a lane holds of one step of one tile ahead of its turn.
template <int NS>
struct Ahead {
    uint32_t w[8];
    uint2 s[NS];
    uint32_t z[NS];
};

// A block's kWarps warps are WK runs of K by kWarps / WK stripes of 16 R channels; a
// cluster of blocks (gridDim.z) splits K again.  Sums of the runs are added in a fixed
// order through (distributed) shared memory.  A block takes every gridDim.x-th set of
// ROWS channels, its x staged once where it fits, and has a set's first weights on
// their way while it adds up the one before.  NS: scales in a step, 1 when the group is
// a multiple of 128, 2 of 64, 4 of 32.
template <int XT, int NT, int R, int WK, bool ZERO, int NS>
__global__ void __launch_bounds__(kWarps * 32, NT == 4 ? 1 : 2) gemv_w4_kernel(const __grid_constant__ GemvArgs a)
{
    constexpr bool BF16 = XT != QNN_F16;
    constexpr int P = Cols<XT>::kParts, TOK = NT * 8 / P, PITCH = NT * 8 + 1;
    constexpr int U = R == 1 ? 4 : 2;  // steps loaded ahead
    constexpr int ROWS = 16 * R * (kWarps / WK);
    extern __shared__ __align__(16) uint8_t smem[];
    float *parts = reinterpret_cast<float *>(smem);  // two of [WK][ROWS][PITCH], used in turn
    uint4 *xs = reinterpret_cast<uint4 *>(smem + kPartBytes<NT, R> * 2);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, j = lane & 3;
    const int run = warp % WK, stripe = warp / WK;
    const int64_t m0 = (int64_t)blockIdx.y * TOK;
    const int toks = (int)min((int64_t)TOK, a.M - m0), cols = toks * P;
    const int splits = gridDim.z, rank = blockIdx.z;
    const int b0 = splits == 1 ? 0 : a.steps * rank / splits,
              b1 = splits == 1 ? a.steps : a.steps * (rank + 1) / splits;
    const int sbytes = a.scale_dt == QNN_F32 ? 64 : 32;  // of one group of a tile
    auto tile_of = [&](int set) { return (set * (kWarps / WK) + stripe) * R; };

    // Weights come to L2 ahead of their use, the first ones while the grid before still
    // runs; nothing is read before that grid's results are there.
    auto prefetch = [&](int set) {
        const int tile = tile_of(set) + lane;
        if (run == 0 && lane < R && tile < a.tiles && b0 < b1)
            prefetch_l2(a.w + ((int64_t)tile * a.steps + b0) * 1024, (b1 - b0) * 1024);
    };

    Ahead<NS> ah[U][R];
    const uint8_t *wp[R], *sp[R], *zp[R];  // the next step to load, and its group's constants
    int gn = 0, left = 0, c0 = 0, c1 = 0;
    auto fetch = [&](Ahead<NS> (&h)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            ldg_stream_v8(wp[r], h[r].w);
            wp[r] += 1024;
        }
#pragma unroll
        for (int q = 0; q < NS; ++q) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h[r].s[q] = load_scales(sp[r], a.scale_dt);
                if constexpr (ZERO) h[r].z[q] = __ldg(reinterpret_cast<const uint16_t *>(zp[r]));
            }
            if (--left == 0) {
                left = a.per_scale;
                if (++gn < a.groups) {  // beyond the last group x is zero
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        sp[r] += sbytes;
                        if constexpr (ZERO) zp[r] += 16;
                    }
                }
            }
        }
    };
    // this warp's run of steps p0 .. p0 + pass_steps of a set, and its first U of them
    auto begin = [&](int set, int p0) {
        const int n = min(p0 + a.pass_steps, b1) - p0, tile0 = tile_of(set);
        c0 = p0 + n * run / WK;
        c1 = tile0 < a.tiles ? p0 + n * (run + 1) / WK : c0;
        gn = (uint32_t)(c0 * NS) / (uint32_t)a.per_scale;
        left = a.per_scale - (c0 * NS - gn * a.per_scale);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t tile = min(tile0 + r, a.tiles - 1);  // a tile beyond N is computed as the last, not stored
            const int64_t at = tile * a.groups + min(gn, a.groups - 1);
            wp[r] = a.w + (tile * a.steps + c0) * 1024 + lane * 32;
            sp[r] = a.scale + at * sbytes + gid * (sbytes / 8);
            if constexpr (ZERO) zp[r] = a.zero + at * 16 + gid * 2;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u < c1) fetch(ah[u]);
    };

    grid_dependency_launch();
    int set = blockIdx.x, p0 = b0, turn = 0;
    bool staged = false;
    prefetch(set);
    grid_dependency_wait();
    begin(set, p0);
    float sum[R][NT][4] = {};
    while (set < a.sets) {
        if (!staged) {
            const int n = min(p0 + a.pass_steps, b1) - p0;
            if (WK == kWarps && a.pass_steps >= b1 - b0) {  // once, each warp the part of x that it alone reads
                for (int tok = 0; tok < toks; ++tok)
                    stage_x<XT>(a, m0 + tok, tok * P, cols, p0 * 128, (c0 - p0) * 16, (c1 - p0) * 16, lane, 32, xs);
                __syncwarp();
            } else {
                __syncthreads();  // xs may still be read
                const int share = 1 << a.lane_bits;  // threads to a row of x
                for (int tok = threadIdx.x >> a.lane_bits; tok < toks; tok += (kWarps * 32) >> a.lane_bits)
                    stage_x<XT>(a, m0 + tok, tok * P, cols, p0 * 128, 0, n * 16, threadIdx.x & (share - 1), share, xs);
                __syncthreads();
            }
            staged = a.pass_steps >= b1 - b0;
        }
        if (p0 == b0 && set + (int)gridDim.x < a.sets) prefetch(set + gridDim.x);

        // columns beyond `cols` are computed as the last one, and not stored
        const uint4 *xc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xc[t] = xs + ((c0 - p0) * 4 * cols + min(t * 8 + gid, cols - 1)) * 4 + j;
        for (int c = c0; c < c1; c += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u >= c1) break;
                float acc[R][NT][4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    constexpr int SPAN = 4 / NS;  // 32-channel parts to a scale
                    uint4 b[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        b[t] = *xc[t];
                        xc[t] += cols * 4;
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const Ahead<NS> &h = ah[u][r];
                        const uint32_t zz = ZERO ? h.z[s / SPAN] : 0x0808u;
                        const ZeroTerm z = zero_term<BF16>(zz & 0xffu, zz >> 8);
                        uint32_t a0[4], a1[4];
                        codes_to_a<BF16>(h.w[2 * s], z, a0);
                        codes_to_a<BF16>(h.w[2 * s + 1], z, a1);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if (s % SPAN == 0)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[r][t][e] = 0.0f;
                            mma16816<BF16>(acc[r][t], a0, b[t].x, b[t].y);
                            mma16816<BF16>(acc[r][t], a1, b[t].z, b[t].w);
                        }
                        if (s % SPAN != SPAN - 1) continue;
                        const float2 sc = scales_f32(h.s[s / SPAN], a.scale_dt);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                sum[r][t][e] = __fmaf_rn(acc[r][t][e], e < 2 ? sc.x : sc.y, sum[r][t][e]);
                    }
                }
                if (c + u + U < c1) fetch(ah[u]);
            }
        }
        const int done = set;
        p0 += a.pass_steps;
        const bool last = p0 >= b1;  // of this set's passes
        if (last) {
            p0 = b0;
            set += gridDim.x;
        }
        if (set < a.sets) begin(set, p0);
        if (!last) continue;

        // the bias of this thread's outputs: kWarps * 32 is a multiple of ROWS
        const int row = threadIdx.x % ROWS;
        const int64_t n = (int64_t)done * ROWS + row;
        const float bias = a.bias && n < a.N ? __ldg(a.bias + n) : 0.0f;
        float *part = parts + turn * (kPartBytes<NT, R> / 4);
        turn ^= 1;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    part[(run * ROWS + (stripe * R + r) * 16 + gid + 8 * (e >> 1)) * PITCH + t * 8 + 2 * j + (e & 1)] =
                        sum[r][t][e];
                    sum[r][t][e] = 0.0f;
                }
        if (splits > 1) cg::this_cluster().sync();
        else __syncthreads();
        constexpr int STEP = kWarps * 32 / ROWS;  // rows of x a block finishes at a time
        for (int tok = threadIdx.x / ROWS + rank * STEP; tok < toks; tok += STEP * splits) {
            if (n >= a.N) break;
            float v = 0.0f;
            for (int q = 0; q < splits; ++q) {
                const float *from =
                    (splits > 1 ? cg::this_cluster().map_shared_rank(part, q) : part) + row * PITCH + tok * P;
#pragma unroll
                for (int p = P - 1; p >= 0; --p)  // the small parts first
#pragma unroll
                    for (int k = 0; k < WK; ++k) v = __fadd_rn(v, from[k * ROWS * PITCH + p]);
            }
            if (a.bias) v = __fadd_rn(v, bias);
            const int64_t at = (m0 + tok) * a.ldy + n;
            if (a.y_dt == QNN_F32) static_cast<float *>(a.y)[at] = v;
            else if (a.y_dt == QNN_F16) static_cast<__half *>(a.y)[at] = from_f32<__half>(v);
            else static_cast<__nv_bfloat16 *>(a.y)[at] = from_f32<__nv_bfloat16>(v);
        }
    }
    if (splits > 1) cg::this_cluster().sync();  // no block leaves while its sums are read
}

// ---- launch ------------------------------------------------------------------------

// shared memory of a block: two blocks on an SM, or one
template <int NT>
constexpr int kMaxSmem = NT == 1 ? 110 << 10 : 200 << 10;

template <int XT, int NT, int R, int WK, bool ZERO, int NS>
qnn_status launch_gemv(GemvArgs a, cudaStream_t s)
{
    constexpr int P = Cols<XT>::kParts, TOK = NT * 8 / P, ROWS = 16 * R * (kWarps / WK);
    const int64_t by = (a.M + TOK - 1) / TOK;
    if (by > 65535) return QNN_ERR_UNSUPPORTED;
    a.sets = (a.tiles + ROWS / 16 - 1) / (ROWS / 16);
    // K split over a cluster while the blocks still run all at once and keep two steps a warp
    const int64_t slots = (NT == 4 ? 1 : 2) * sm_count();
    int splits = 1;
    if (WK < kWarps)
        while (splits < 4 && a.sets * by * splits * 2 <= slots && a.steps >= 4 * splits * WK) splits *= 2;
    const int cols = (int)std::min<int64_t>(a.M, TOK) * P, span = (a.steps + splits - 1) / splits;
    // x in passes of what kMaxSmem holds (two blocks on an SM); a step is 256 bytes a column
    constexpr int PARTS = 2 * kPartBytes<NT, R>;
    a.pass_steps = std::min(span, (kMaxSmem<NT> - PARTS) / (cols * 256));
    a.lane_bits = 5;
    while (a.lane_bits < 8 && (16 * a.pass_steps) >> a.lane_bits > 1) ++a.lane_bits;
    const int smem = PARTS + a.pass_steps * cols * 256;
    auto kern = gemv_w4_kernel<XT, NT, R, WK, ZERO, NS>;
    static std::atomic<uint64_t> opted_in{0};  // devices on which the kernel may take kMaxSmem
    if (smem > (48 << 10) && !opt_in_smem(kern, kMaxSmem<NT>, opted_in)) return QNN_ERR_CUDA;
    // equal numbers of sets for the blocks that run at once
    const int64_t most = std::max<int64_t>(slots / (by * splits), 1), rounds = (a.sets + most - 1) / most;
    const int64_t bx = (a.sets + rounds - 1) / rounds;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)bx, (unsigned)by, (unsigned)splits);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {1, 1, (unsigned)splits};
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return QNN_ERR_CUDA;
    }
    return launch_status();
}

template <int XT, int NT, int R, int WK, bool ZERO>
qnn_status launch_gemv_group(GemvArgs a, int group, cudaStream_t s)
{
    a.per_scale = group % 128 == 0 ? group / 128 : group % 64 == 0 ? group / 64 : group / 32;
    if (group % 128 == 0) return launch_gemv<XT, NT, R, WK, ZERO, 1>(a, s);
    if (group % 64 == 0) return launch_gemv<XT, NT, R, WK, ZERO, 2>(a, s);
    return launch_gemv<XT, NT, R, WK, ZERO, 4>(a, s);
}

template <int XT, int NT, int R, int WK>
qnn_status launch_gemv_zero(const GemvArgs &a, int group, cudaStream_t s)
{
    return a.zero ? launch_gemv_group<XT, NT, R, WK, true>(a, group, s)
                  : launch_gemv_group<XT, NT, R, WK, false>(a, group, s);
}

template <int XT>
qnn_status launch_gemv_type(const GemvArgs &a, int group, cudaStream_t s)
{
    const int64_t cols = a.M * Cols<XT>::kParts;
    if (cols > 16) return launch_gemv_zero<XT, 4, 2, 2>(a, group, s);
    if (cols > 8) return launch_gemv_zero<XT, 2, 2, 4>(a, group, s);
    // two tiles a warp as soon as that still gives every SM a block
    const bool two = a.tiles > 2 * sm_count();
    return two ? launch_gemv_zero<XT, 1, 2, 8>(a, group, s) : launch_gemv_zero<XT, 1, 1, 8>(a, group, s);
}

int grid_for(int64_t work)
{
    return (int)std::max<int64_t>(1, std::min<int64_t>((work + 255) / 256, (int64_t)sm_count() * 8));
}

}  // namespace
}  // namespace qnn

extern "C" size_t qnn_gemv_w4_packed_bytes(const qnn_w4_geom *g)
{
    qnn::W4Image im;
    return qnn::w4_image(g, &im) ? im.total : 0;
}

extern "C" qnn_status qgemv_prepack_w4(const void *W, const void *scale, const int32_t *zero_point,
                                       const qnn_w4_geom *g, void *W_packed, qnn_stream_t stream)
{
    using namespace qnn;
    W4Image im;
    if (!w4_image(g, &im)) return QNN_ERR_INVALID_ARG;
    if (!W || !scale || !W_packed || (zero_point != nullptr) != (g->w_dt == QNN_U4)) return QNN_ERR_INVALID_ARG;
    if (!aligned16(W) || !aligned16(scale) || !aligned_image(W_packed) || (zero_point && !aligned16(zero_point)))
        return QNN_ERR_ALIGNMENT;
    uint32_t *st = status_word();
    if (!st) return QNN_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t *out = static_cast<uint8_t *>(W_packed);
    const int64_t words = im.tiles * im.steps * 256, total = im.tiles * im.groups * 16;
    prepack_w4_kernel<<<grid_for(words), 256, 0, s>>>(static_cast<const uint8_t *>(W), g->N, g->K, im.steps, words,
                                                      g->w_dt == QNN_S4, reinterpret_cast<uint32_t *>(out));
    const qnn_status first = launch_status();
    if (first != QNN_OK) return first;
    if (g->scale_dt == QNN_F32)
        prepack_w4_scale_kernel<<<grid_for(total), 256, 0, s>>>(
            static_cast<const uint32_t *>(scale), zero_point, (int64_t)g->N, im.groups, total,
            reinterpret_cast<uint32_t *>(out + im.scale_off), out + im.zero_off, st);
    else
        prepack_w4_scale_kernel<<<grid_for(total), 256, 0, s>>>(
            static_cast<const uint16_t *>(scale), zero_point, (int64_t)g->N, im.groups, total,
            reinterpret_cast<uint16_t *>(out + im.scale_off), out + im.zero_off, st);
    return launch_status();
}

extern "C" qnn_status qgemv_w4(const void *x, qnn_dtype x_dt, int64_t ldx, const void *W_packed,
                               const qnn_w4_geom *g, int64_t M, const float *bias, void *y, qnn_dtype y_dt,
                               int64_t ldy, qnn_stream_t stream)
{
    using namespace qnn;
    W4Image im;
    if (!w4_image(g, &im) || M < 0) return QNN_ERR_INVALID_ARG;
    if (!is_float_dt(x_dt) || (y_dt != x_dt && y_dt != QNN_F32)) return QNN_ERR_UNSUPPORTED;
    if (ldx == 0) ldx = g->K;
    if (ldy == 0) ldy = g->N;
    if (ldx < g->K || ldy < g->N) return QNN_ERR_INVALID_ARG;
    if (M == 0) return QNN_OK;
    if (!x || !W_packed || !y) return QNN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned_image(W_packed) || !aligned16(y) || (bias && !aligned16(bias)))
        return QNN_ERR_ALIGNMENT;
    const uint8_t *w = static_cast<const uint8_t *>(W_packed);
    GemvArgs a{};
    a.x = x;
    a.w = w;
    a.scale = w + im.scale_off;
    a.zero = g->w_dt == QNN_U4 ? w + im.zero_off : nullptr;
    a.bias = bias;
    a.y = y;
    a.ldx = ldx;
    a.ldy = ldy;
    a.M = M;
    a.N = g->N;
    a.K = g->K;
    a.tiles = (int)im.tiles;
    a.steps = (int)im.steps;
    a.groups = (int)im.groups;
    a.y_dt = y_dt;
    a.scale_dt = g->scale_dt;
    a.vec = ldx * float_bytes(x_dt) % 16 == 0;
    cudaStream_t s = (cudaStream_t)stream;
    switch (x_dt) {
    case QNN_F32: return launch_gemv_type<QNN_F32>(a, g->group, s);
    case QNN_F16: return launch_gemv_type<QNN_F16>(a, g->group, s);
    default: return launch_gemv_type<QNN_BF16>(a, g->group, s);
    }
}
