// qnn_gemv.cu -- qgemv_w4: a few rows of activations times 4-bit weights with
// group scales (the weight-only linear layer at decoding sizes).
//
//   y[m][n] = bias[n] + sum_g s[n][g] sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weights are read once and are nearly all the bytes, so the op is bound by
// the weight stream; what has to be kept off that path is the arithmetic on the
// codes, about three issue slots per weight at full bandwidth.  Converting each code
// to fp32 and multiplying it on the CUDA cores takes that many for one row of x and
// more for two; here the codes become f16 or bf16 integers two at a time and the
// products run on the tensor cores (mma.sync m16n8k16: 16 output channels x 8
// columns of x), about 1.2 slots per weight for up to 8 rows of x.
//
// The image (prepack): per tile of 16 output channels and step of 64 input
// channels, 512 bytes = one 16-byte load per lane.  A 32-bit word of lane (g, j)
// (g = lane / 4, j = lane % 4) holds channels n = g and g + 8 at four consecutive
// k: nibbles at bits 0/16: (g; k, k+1), 4/20: (g+8; k, k+1), 8/24: (g; k+2, k+3),
// 12/28: (g+8; k+2, k+3), which are the four registers of the MMA's A fragment.
// Word w of the lane covers k = 32 (w / 2) + 8 j + 4 (w % 2): as the order of K is
// free, a lane's 8 values of x for two MMAs are then one contiguous load.
// Behind the codes: the scales [tile][group][16], then (U4) the zero points, bytes.
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include "qnn_float.cuh"
#include "qnn_internal.h"
#include "qnn_ptx.cuh"

namespace qnn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;

struct W4Image {
    int64_t tiles, chunks, groups;  // ceil(N / 16), ceil(K / 64), ceil(K / group)
    size_t scale_off, zero_off, total;
};

bool w4_image(const qnn_w4_geom *g, W4Image *im)
{
    if (!g || g->N <= 0 || g->K <= 0 || g->K > (1 << 30) || g->K % 2 != 0 || g->group <= 0 || g->group % 32 != 0) return false;
    if ((g->w_dt != QNN_S4 && g->w_dt != QNN_U4) || !is_float_dt(g->scale_dt)) return false;
    im->tiles = ((int64_t)g->N + 15) / 16;
    im->chunks = ((int64_t)g->K + 63) / 64;
    im->groups = ((int64_t)g->K + g->group - 1) / g->group;
    im->scale_off = (size_t)im->tiles * im->chunks * 512;
    im->zero_off = im->scale_off + (size_t)im->tiles * im->groups * 16 * float_bytes(g->scale_dt);
    im->total = im->zero_off + (g->w_dt == QNN_U4 ? (size_t)im->tiles * im->groups * 16 : 0);
    return true;
}

// ---- prepack -----------------------------------------------------------------------

// One thread per word of the image; a code outside [N, K) is its zero point.
// Codes are stored offset: q + 8 for S4, so that both types are u4 with a zero point.
__global__ void __launch_bounds__(256) prepack_w4_kernel(const uint8_t *__restrict__ W, int64_t N, int64_t K,
                                                         int64_t chunks, int64_t words, int is_signed,
                                                         uint32_t *__restrict__ out)
{
    const int64_t pitch = K / 2;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int w = (int)(i & 3), lane = (int)(i >> 2) & 31;
        const int64_t chunk = (i >> 7) % chunks, tile = (i >> 7) / chunks;
        const int64_t k = chunk * 64 + (w >> 1) * 32 + (lane & 3) * 8 + (w & 1) * 4;
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

// scales (copied bit for bit) and zero points, [N, G] -> [tile][g][16]
template <typename T>
__global__ void __launch_bounds__(256) prepack_w4_scale_kernel(const T *__restrict__ scale,
                                                               const int32_t *__restrict__ zero, int64_t N,
                                                               int64_t G, int64_t total, T *__restrict__ out,
                                                               uint8_t *__restrict__ zout, uint32_t *status)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t n = (i >> 4) / G * 16 + (i & 15), g = (i >> 4) % G;
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
    const uint8_t *scale;  // [tile][G][16] of scale_dt
    const uint8_t *zero;   // [tile][G][16], or nullptr
    const float *bias;
    void *y;
    int64_t ldx, ldy, M;
    int N, K, chunks, groups, group_subs;  // group_subs: group / 32
    int scale_dt, y_dt;
    int vec;  // rows of x start on 16-byte boundaries
};

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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

__device__ __forceinline__ uint32_t hfma2_u32(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t bfma2_u32(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The zero points of a lane's two channels as the addends of the code conversion.
struct ZeroTerm {
    uint32_t lo, hi;
};

// f16: 0x6400 | q is 1024 + q, and 0x6400 | 16 q is 1024 + 16 q, which a multiply by
// 1/16 takes to 64 + q.  bf16: 0x4300 | q is 128 + q (the nibbles shifted down, as
// 128 + 16 q would not fit its 8 bits).  Subtracting magic + z is exact: |q - z| <= 15.
template <bool BF16>
__device__ __forceinline__ ZeroTerm zero_term(uint32_t z_lo, uint32_t z_hi)
{
    ZeroTerm t;
    if constexpr (BF16) {
        t.lo = 0xc300c300u | z_lo * 0x10001u;            // -(128 + z)
        t.hi = 0xc300c300u | z_hi * 0x10001u;
    } else {
        t.lo = 0xe400e400u | z_lo * 0x10001u;            // -(1024 + z)
        t.hi = 0xd400d400u | (z_hi << 4) * 0x10001u;     // -(64 + z)
    }
    return t;
}

template <bool BF16>
__device__ __forceinline__ void codes_to_a(uint32_t w, const ZeroTerm &z, uint32_t (&a)[4])
{
    if constexpr (BF16) {
        const uint32_t one = 0x3f803f80u;
        a[0] = bfma2_u32(nib(w, 0x000f000fu, 0x43004300u), one, z.lo);
        a[1] = bfma2_u32(nib(w >> 4, 0x000f000fu, 0x43004300u), one, z.hi);
        a[2] = bfma2_u32(nib(w >> 8, 0x000f000fu, 0x43004300u), one, z.lo);
        a[3] = bfma2_u32(nib(w >> 12, 0x000f000fu, 0x43004300u), one, z.hi);
    } else {
        const uint32_t one = 0x3c003c00u, sixteenth = 0x2c002c00u, v = w >> 8;
        a[0] = hfma2_u32(nib(w, 0x000f000fu, 0x64006400u), one, z.lo);
        a[1] = hfma2_u32(nib(w, 0x00f000f0u, 0x64006400u), sixteenth, z.hi);
        a[2] = hfma2_u32(nib(v, 0x000f000fu, 0x64006400u), one, z.lo);
        a[3] = hfma2_u32(nib(v, 0x00f000f0u, 0x64006400u), sixteenth, z.hi);
    }
}

// Column of the B operand -> (row of x, part).  fp32 rows take three columns: x is the
// exact sum of three bf16, its leading 8 bits, the next 8 and the rest, each cut (not
// rounded, so that none overflows); infinities and NaN go into the first alone.
template <int XT>
struct Cols {
    static constexpr int kParts = XT == QNN_F32 ? 3 : 1;
};

__device__ __forceinline__ uint32_t bf16_part(float v, int part)
{
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7f800000u) == 0x7f800000u)
        return part ? 0u : (u & 0x007fffffu) ? 0x7fc0u : u >> 16;
    float r = v;
    uint32_t top = u & 0xffff0000u;
    for (int p = 0; p < part; ++p) {
        r = __fsub_rn(r, __uint_as_float(top));  // exact
        top = __float_as_uint(r) & 0xffff0000u;
    }
    return top >> 16;
}

// The lane's 8 values of x at k .. k+7 as four pairs; zero beyond K or for a column
// without a row (xr = nullptr).
template <int XT>
__device__ __forceinline__ uint4 load_x(const void *xr, int part, int k, int K, int vec)
{
    uint32_t o[4] = {0, 0, 0, 0};
    if (xr && k < K) {
        if constexpr (XT == QNN_F32) {
            const float *p = static_cast<const float *>(xr) + k;
            float v[8];
            if (vec && k + 8 <= K) {
                const float4 a = __ldg(reinterpret_cast<const float4 *>(p)),
                             b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = k + i < K ? __ldg(p + i) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = bf16_part(v[2 * i], part) | bf16_part(v[2 * i + 1], part) << 16;
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(xr) + k;
            if (vec && k + 8 <= K) return __ldg(reinterpret_cast<const uint4 *>(p));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < K) o[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float load_scale(const uint8_t *p, int dt, int64_t i)
{
    if (dt == QNN_F32) return __ldg(reinterpret_cast<const float *>(p) + i);
    const uint16_t u = __ldg(reinterpret_cast<const uint16_t *>(p) + i);
    return dt == QNN_F16 ? __half2float(__ushort_as_half(u)) : __uint_as_float((uint32_t)u << 16);
}

// One block per tile of 16 channels and 8 NT columns; its warps take equal runs of
// K and their sums are added in a fixed order through shared memory.
template <int XT, int NT, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32) gemv_w4_kernel(const __grid_constant__ GemvArgs a)
{
    constexpr bool BF16 = XT != QNN_F16;
    constexpr int P = Cols<XT>::kParts, TOK = NT * 8 / P;  // rows of x per block
    __shared__ float part[kWarps][16][NT * 8 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, j = lane & 3;
    const int64_t tile = blockIdx.x, m0 = (int64_t)blockIdx.y * TOK;

    const void *xr[NT];
    int xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = t * 8 + gid, tok = col / P;
        xp[t] = col % P;
        xr[t] = tok < TOK && m0 + tok < a.M
                    ? static_cast<const uint8_t *>(a.x) + (m0 + tok) * a.ldx * (XT == QNN_F32 ? 4 : 2)
                    : nullptr;
    }
    const int c0 = (int)((int64_t)a.chunks * warp / kWarps), c1 = (int)((int64_t)a.chunks * (warp + 1) / kWarps);
    const uint4 *wp = reinterpret_cast<const uint4 *>(a.w) + (tile * a.chunks) * 32 + lane;
    const int64_t srow = tile * a.groups * 16 + gid;

    float sum[NT][4] = {}, acc[NT][4] = {};
    int g = 2 * c0 / a.group_subs, left = a.group_subs - 2 * c0 % a.group_subs;
    ZeroTerm z = zero_term<BF16>(8, 8);
    float s_lo = 0.0f, s_hi = 0.0f;
    auto enter = [&]() {  // the constants of group g (the last one's beyond K)
        const int64_t i = srow + (int64_t)min(g, a.groups - 1) * 16;
        s_lo = load_scale(a.scale, a.scale_dt, i);
        s_hi = load_scale(a.scale, a.scale_dt, i + 8);
        if constexpr (ZERO) z = zero_term<BF16>(__ldg(a.zero + i), __ldg(a.zero + i + 8));
    };
    auto leave = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[t][e] = __fmaf_rn(acc[t][e], e < 2 ? s_lo : s_hi, sum[t][e]);
                acc[t][e] = 0.0f;
            }
    };
    if (c0 < c1) enter();
    for (int c = c0; c < c1; ++c) {
        const uint4 w4 = __ldcs(wp + (int64_t)c * 32);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (left == 0) {
                leave();
                ++g;
                left = a.group_subs;
                enter();
            }
            --left;
            uint32_t a0[4], a1[4];
            codes_to_a<BF16>(w[2 * s], z, a0);
            codes_to_a<BF16>(w[2 * s + 1], z, a1);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 b = load_x<XT>(xr[t], xp[t], c * 64 + s * 32 + j * 8, a.K, a.vec);
                mma16816<BF16>(acc[t], a0, b.x, b.y);
                mma16816<BF16>(acc[t], a1, b.z, b.w);
            }
        }
    }
    leave();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][gid + 8 * (e >> 1)][t * 8 + 2 * j + (e & 1)] = sum[t][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * TOK; i += kWarps * 32) {
        const int r = i & 15, tok = i >> 4;
        const int64_t n = tile * 16 + r, m = m0 + tok;
        if (n >= a.N || m >= a.M) continue;
        float v = 0.0f;
#pragma unroll
        for (int p = P - 1; p >= 0; --p)  // the small parts first
            for (int k = 0; k < kWarps; ++k) v = __fadd_rn(v, part[k][r][tok * P + p]);
        if (a.bias) v = __fadd_rn(v, __ldg(a.bias + n));
        const int64_t at = m * a.ldy + n;
        if (a.y_dt == QNN_F32) static_cast<float *>(a.y)[at] = v;
        else if (a.y_dt == QNN_F16) static_cast<__half *>(a.y)[at] = from_f32<__half>(v);
        else static_cast<__nv_bfloat16 *>(a.y)[at] = from_f32<__nv_bfloat16>(v);
    }
}

template <int XT, int NT>
qnn_status launch_gemv(const GemvArgs &a, int64_t tiles, cudaStream_t s)
{
    constexpr int TOK = NT * 8 / Cols<XT>::kParts;
    const int64_t by = (a.M + TOK - 1) / TOK;
    if (by > 65535) return QNN_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)tiles, (unsigned)by);
    if (a.zero) gemv_w4_kernel<XT, NT, true><<<grid, kWarps * 32, 0, s>>>(a);
    else gemv_w4_kernel<XT, NT, false><<<grid, kWarps * 32, 0, s>>>(a);
    return launch_status();
}

template <int XT>
qnn_status launch_gemv_xt(const GemvArgs &a, int64_t tiles, cudaStream_t s)
{
    const int64_t cols = a.M * Cols<XT>::kParts;
    if (cols <= 8) return launch_gemv<XT, 1>(a, tiles, s);
    if (cols <= 16) return launch_gemv<XT, 2>(a, tiles, s);
    return launch_gemv<XT, 4>(a, tiles, s);
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
    if (!aligned16(W) || !aligned16(scale) || !aligned16(W_packed) || (zero_point && !aligned16(zero_point)))
        return QNN_ERR_ALIGNMENT;
    uint32_t *st = status_word();
    if (!st) return QNN_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t *out = static_cast<uint8_t *>(W_packed);
    const int64_t words = im.tiles * im.chunks * 128, total = im.tiles * im.groups * 16;
    prepack_w4_kernel<<<grid_for(words), 256, 0, s>>>(static_cast<const uint8_t *>(W), g->N, g->K, im.chunks, words,
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
    if (!aligned16(x) || !aligned16(W_packed) || !aligned16(y) || (bias && !aligned16(bias)))
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
    a.chunks = (int)im.chunks;
    a.groups = (int)im.groups;
    a.group_subs = g->group / 32;
    a.scale_dt = g->scale_dt;
    a.y_dt = y_dt;
    a.vec = ldx * float_bytes(x_dt) % 16 == 0;
    cudaStream_t s = (cudaStream_t)stream;
    switch (x_dt) {
    case QNN_F32: return launch_gemv_xt<QNN_F32>(a, im.tiles, s);
    case QNN_F16: return launch_gemv_xt<QNN_F16>(a, im.tiles, s);
    default: return launch_gemv_xt<QNN_BF16>(a, im.tiles, s);
    }
}
