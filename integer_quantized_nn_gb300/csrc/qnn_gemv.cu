// qnn_gemv.cu -- qgemv_w4: a few rows of activations times 4-bit weights with
// group scales (the weight-only linear layer at decoding sizes).
//
//   y[m][n] = bias[n] + sum_g s[n][g] sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weights are read once and are nearly all the bytes, so the op is bound by the
// weight stream: 23 bytes, 47 codes, a clock and SM.  The SM's integer pipe does 64
// operations a clock, which is not much more, so what is done to a code decides.  The
// codes become f16 or bf16 integers two at a time (9 operations for 8 codes in f16, 11 in
// bf16) and the products run on the tensor cores (mma.sync m16n8k16: 16 output channels
// x 8 columns of x); multiplying on the CUDA cores takes more than two operations a code
// for one row of x alone.  This kernel is for up to 8 columns; qnn_gemv_columns.cu has
// the one for more.
//
// Measured (one row, groups of 128), over weights that L2 cannot hold and, in brackets, over
// three copies in turn, of which it can keep some or all: 8192 x 8192 bf16 9.8 us [9.1], 3.7
// TB/s, 0.54 of a copy's bandwidth; 4096 x 4096 f16 4.3 [3.8]; 1024 x 1024 (groups of 64) 2.4
// [2.2]; 131072 x 4096 bf16 64 us, 4.3 TB/s.  That is 2 to 5 us beyond the bytes, at 131072
// channels 23.  8192 x 8192 makes 256 blocks for 152 SMs: an SM's issue is 24 to 49 % busy, by
// how many blocks it has.  Shifting codes on the multiplier pipe (mul.hi) was slower (13.4 us
// to 10.9 at that stage).
//
// The image (prepack): per tile of 16 output channels and step of 128 input
// channels, 1024 bytes, 32 a lane.  A 32-bit word of lane (g, j) (g = lane / 4, j =
// lane % 4) holds channels n = g and g + 8 at four consecutive k: nibbles at bits
// 0/16: (g; k, k+1), 4/20: (g+8; k, k+1), 8/24: (g; k+2, k+3), 12/28: (g+8; k+2, k+3),
// the four registers of the MMA's A fragment.  Word w of the lane covers k =
// 32 (w / 2) + 8 j + 4 (w % 2): the order of K is free, and so a lane's 8 values of x
// for two MMAs are contiguous.  Behind the codes: the scales [tile][group][8][2]
// (channels n, n + 8), then (U4) the zero points in the same order, bytes.
#include "qnn_gemv.cuh"

namespace qnn {
namespace {

constexpr int kWarps = 8;

// one buffer of the warps' sums: [runs][channels of a set][columns, padded]
constexpr int kPitch = 9;
template <int R>
constexpr int kPartBytes = kWarps * 16 * R * kPitch * 4;

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

// Pieces i0 .. i1 - 1 of row `row` of x (at k = 8 i), by one warp, to shared memory as B
// fragments, [32 channels][column][j]; zero beyond K.
template <int XT>
__device__ __forceinline__ void stage_x(const GemvArgs &a, int64_t row, int col, int cols, int i0, int i1, int lane,
                                        uint4 *xs)
{
    constexpr int W = XT == QNN_F32 ? 2 : 1;  // 16-byte words of a piece
    const uint8_t *p = static_cast<const uint8_t *>(a.x) + row * a.ldx * (2 * W);
    const int end = a.K, whole = a.align == 16 ? min(i1, end >> 3) : i0;
#pragma unroll 4
    for (int i = i0 + lane; i < whole; i += 32) {
        const uint4 *v = reinterpret_cast<const uint4 *>(p) + (int64_t)i * W;
        const uint4 u = load_input(v);
        put_piece<XT>(u, W == 2 ? load_input(v + W - 1) : u, xs + ((i >> 2) * cols + col) * 4 + (i & 3));
    }
    // rows off 16-byte boundaries and the ragged end: value by value
#pragma unroll 8
    for (int e = max(whole, i0) * 8 + lane; e < i1 * 8; e += 32) {
        uint16_t *out = reinterpret_cast<uint16_t *>(xs + ((e >> 5) * cols + col) * 4 + (e >> 3 & 3)) + (e & 7);
        if constexpr (W == 2) {
            uint32_t v[3];
            bf16_parts(e < end ? load_input(reinterpret_cast<const float *>(p) + e) : 0.0f, v);
#pragma unroll
            for (int q = 0; q < 3; ++q) out[32 * q] = (uint16_t)v[q];
        } else {
            *out = e < end ? load_input(reinterpret_cast<const uint16_t *>(p) + e) : (uint16_t)0;
        }
    }
}

// What a lane holds of one step of one tile ahead of its turn.
template <int NS>
struct Ahead {
    uint32_t w[8];
    uint2 s[NS];
    uint32_t z[NS];
};

// A block's warps are kWarps runs of K of the same 16 R channels; their sums are added in
// a fixed order through shared memory.  A warp stages the part of x that it alone reads,
// once.  A block takes every gridDim.x-th set of 16 R channels, and has a set's first
// weights on their way while it adds up the one before.  NS: scales in a step, 1 when the
// group is a multiple of 128, 2 of 64, 4 of 32.
template <int XT, int R, bool ZERO, int NS>
__global__ void __launch_bounds__(kWarps * 32, 2) gemv_w4_kernel(const __grid_constant__ GemvArgs a)
{
    constexpr bool BF16 = XT != QNN_F16;
    constexpr int P = Cols<XT>::kParts, ROWS = 16 * R, U = R == 1 ? 4 : 2;  // U: steps loaded ahead
    extern __shared__ __align__(16) uint8_t smem[];
    float *parts = reinterpret_cast<float *>(smem);  // two of [kWarps][ROWS][kPitch], used in turn
    uint4 *xs = reinterpret_cast<uint4 *>(smem + kPartBytes<R> * 2);
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, gid = lane >> 2, j = lane & 3;
    const int toks = (int)a.M, cols = toks * P;
    const int c0 = a.steps * run / kWarps, c1 = a.steps * (run + 1) / kWarps;  // this warp's steps
    const int sbytes = a.scale_dt == QNN_F32 ? 64 : 32;                         // of one group of a tile

    // Weights come to L2 ahead of their use, the first ones while the grid before still
    // runs; nothing is read before that grid's results are there.
    auto prefetch = [&](int set) {
        const int tile = set * R + lane;
        if (run == 0 && lane < R && tile < a.tiles) prefetch_l2(a.w + (int64_t)tile * a.steps * 1024, a.steps * 1024);
    };

    Ahead<NS> ah[U][R];
    const uint8_t *wp[R], *sp[R], *zp[R];  // the next step to load, and its group's constants
    int gn = 0, left = 0;
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
                if constexpr (ZERO) h[r].z[q] = load_input(reinterpret_cast<const uint16_t *>(zp[r]));
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
    // the first steps of a set
    auto begin = [&](int set) {
        gn = (uint32_t)(c0 * NS) / (uint32_t)a.per_scale;
        left = a.per_scale - (c0 * NS - gn * a.per_scale);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t tile = min(set * R + r, a.tiles - 1);  // a tile beyond N is computed as the last, not stored
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
    prefetch(blockIdx.x);
    grid_dependency_wait();
    begin(blockIdx.x);
    for (int tok = 0; tok < toks; ++tok) stage_x<XT>(a, tok, tok * P, cols, c0 * 16, c1 * 16, lane, xs);
    __syncwarp();
    int turn = 0;
    for (int set = blockIdx.x; set < a.sets; set += gridDim.x) {
        if (set + (int)gridDim.x < a.sets) prefetch(set + gridDim.x);
        float sum[R][4] = {};
        // columns beyond `cols` are computed as the last one, and not stored
        const uint4 *xc = xs + (c0 * 4 * cols + min(gid, cols - 1)) * 4 + j;
        for (int c = c0; c < c1; c += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u >= c1) break;
                float acc[R][4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    constexpr int SPAN = 4 / NS;  // 32-channel parts to a scale
                    const uint4 b = *xc;
                    xc += cols * 4;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const Ahead<NS> &h = ah[u][r];
                        const uint32_t zz = ZERO ? h.z[s / SPAN] : 0x0808u;
                        const ZeroTerm z = zero_term<BF16>(zz & 0xffu, zz >> 8);
                        uint32_t a0[4], a1[4];
                        codes_to_a<BF16>(h.w[2 * s], z, a0);
                        codes_to_a<BF16>(h.w[2 * s + 1], z, a1);
                        if (s % SPAN == 0)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[r][e] = 0.0f;
                        mma16816<BF16>(acc[r], a0, b.x, b.y);
                        mma16816<BF16>(acc[r], a1, b.z, b.w);
                        if (s % SPAN != SPAN - 1) continue;
                        const float2 sc = scales_f32(h.s[s / SPAN], a.scale_dt);
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[r][e] = __fmaf_rn(acc[r][e], e < 2 ? sc.x : sc.y, sum[r][e]);
                    }
                }
                if (c + u + U < c1) fetch(ah[u]);
            }
        }
        if (set + (int)gridDim.x < a.sets) begin(set + gridDim.x);

        // the bias of this thread's outputs: kWarps * 32 is a multiple of ROWS
        const int row = threadIdx.x % ROWS;
        const int64_t n = (int64_t)set * ROWS + row;
        const float bias = a.bias && n < a.N ? load_input(a.bias + n) : 0.0f;
        float *part = parts + turn * (kPartBytes<R> / 4);
        turn ^= 1;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[(run * ROWS + r * 16 + gid + 8 * (e >> 1)) * kPitch + 2 * j + (e & 1)] = sum[r][e];
        __syncthreads();  // and part is written again behind the next set's barrier only
        for (int tok = threadIdx.x / ROWS; tok < toks && n < a.N; tok += kWarps * 32 / ROWS) {
            float v = 0.0f;
            const float *from = part + row * kPitch + tok * P;
#pragma unroll
            for (int p = P - 1; p >= 0; --p)  // the small parts first
#pragma unroll
                for (int k = 0; k < kWarps; ++k) v = __fadd_rn(v, from[k * ROWS * kPitch + p]);
            if (a.bias) v = __fadd_rn(v, bias);
            store_y(a, tok * a.ldy + n, v);
        }
    }
}

// ---- launch ------------------------------------------------------------------------

constexpr int kMaxSmem = 110 << 10;  // of a block, two of them on an SM

// Shared memory of a block that holds x whole.
template <int R>
int64_t gemv_smem(const GemvArgs &a, int parts)
{
    return 2 * kPartBytes<R> + a.M * parts * 256 * (int64_t)a.steps;
}

template <int XT, int R, bool ZERO, int NS>
qnn_status launch_gemv(GemvArgs a, cudaStream_t s)
{
    auto kern = gemv_w4_kernel<XT, R, ZERO, NS>;
    const int smem = (int)gemv_smem<R>(a, Cols<XT>::kParts);
    static std::atomic<uint64_t> opted_in{0};  // devices on which the kernel may take kMaxSmem
    if (smem > (48 << 10) && !opt_in_smem(kern, kMaxSmem, opted_in)) return QNN_ERR_CUDA;
    a.sets = (a.tiles + R - 1) / R;
    // equal numbers of sets for the blocks that run at once
    const int slots = 2 * sm_count(), rounds = (a.sets + slots - 1) / slots;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.sets + rounds - 1) / rounds));
    cfg.blockDim = dim3(kWarps * 32);
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

template <int XT, int R, bool ZERO>
qnn_status launch_gemv_group(GemvArgs a, int group, cudaStream_t s)
{
    a.per_scale = group % 128 == 0 ? group / 128 : group % 64 == 0 ? group / 64 : group / 32;
    if (group % 128 == 0) return launch_gemv<XT, R, ZERO, 1>(a, s);
    if (group % 64 == 0) return launch_gemv<XT, R, ZERO, 2>(a, s);
    return launch_gemv<XT, R, ZERO, 4>(a, s);
}

template <int XT>
qnn_status launch_gemv_type(const GemvArgs &a, int group, cudaStream_t s)
{
    constexpr int P = Cols<XT>::kParts;
    // x has to fit beside the sums; 8 rows of 8192 bf16 do not, and take 17.5 us by columns (4
    // rows take 10.5 here, both 1 to 2 us less with some of the weights in L2)
    if (a.M * P > 8 || gemv_smem<2>(a, P) > kMaxSmem) return launch_gemv_columns(a, XT, group, s);
    // two tiles a warp share the loads of x and a set's fixed costs, as soon as they leave
    // every SM two blocks (bf16, one row: 8192 x 8192 takes 9.2 us with two, 10.9 with one;
    // 4096 x 4096 takes 5.6 and 4.1)
    if (a.tiles > 2 * sm_count())
        return a.zero ? launch_gemv_group<XT, 2, true>(a, group, s) : launch_gemv_group<XT, 2, false>(a, group, s);
    return a.zero ? launch_gemv_group<XT, 1, true>(a, group, s) : launch_gemv_group<XT, 1, false>(a, group, s);
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
    // the passes are a grid's y; ahead of the products of M below, which it keeps in range
    if (M > 65535 * (int64_t)(kMaxCols / (x_dt == QNN_F32 ? Cols<QNN_F32>::kParts : 1))) return QNN_ERR_UNSUPPORTED;
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
    const int64_t pitch = ldx * float_bytes(x_dt);
    a.align = pitch % 16 == 0 ? 16 : pitch % 8 == 0 ? 8 : pitch % 4 == 0 ? 4 : 2;
    a.status = status_word();
    if (!a.status) return QNN_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    switch (x_dt) {
    case QNN_F32: return launch_gemv_type<QNN_F32>(a, g->group, s);
    case QNN_F16: return launch_gemv_type<QNN_F16>(a, g->group, s);
    default: return launch_gemv_type<QNN_BF16>(a, g->group, s);
    }
}
