// qnn_blocknorm.cu -- q_block_norm: the norm after a block, its gate and residual scale, the
// residual add and the norm before the next block, row by row in one pass.
//
//   p  = norm_post(y)      r' = a r + b gate p      h = norm_pre(r')
//
// norm: x^ = x / sqrt(mean(x^2) + eps)  (RMS)  or  (x - mean) / sqrt(var + eps)
// (LAYER), then gamma x^ + beta.
//
// Bound by the bytes of the rows.  A row is read once and lives in registers to its
// writes: one warp holds rows of up to 1024 columns (through a ring; 256 by direct loads,
// 512 where many rows are off 16-byte boundaries), a block longer ones.  Statistics are
// fp32, the variance from the centred values (a second reduction over registers, not over
// memory).  h is formed from r' before r' is rounded to its own type.
//
// Many rows on 16-byte boundaries: the rows to come are on their way to shared memory
// by bulk copies while one is computed (the copies in flight, not registers, are what
// covers the memory's latency).  Few rows, and rows off those boundaries: direct loads.
//
// Measured, over data that L2 cannot hold: 8192 x 4096 bf16 to s8 codes 41.3 us, 5.7 TB/s
// (0.84 of a copy's bandwidth); 12608 x 768, fp32 stream, LAYER norms with betas, a gate per
// 197 rows: 28.6 us, 4.1 TB/s (issue 49 %, the stalls waits on global and shared loads); 777 x
// 1003 f16 7.7 us (5.9 out of L2); one row of 4096 2.4 us; 2048 x 16384 bf16 61 us, 4.4 TB/s
// (no ring, 100 bytes of spills a thread).  Odd widths load element by element: 8192 x 2003
// bf16 71 us, 1.9 TB/s (through a ring 92); 2048 x 16385 207 us, 1.3 TB/s.
#include "qnn_blocknorm.cuh"

namespace qnn {
namespace {

constexpr int kWarpRows = 4;  // warps (rows) per block where a warp holds a row

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

// rint(t) of |t| <= 128 in the low byte: adding 1.5 2^23 leaves the integer in the low
// bits of the sum, rounded half to even.
__device__ __forceinline__ uint32_t low_int(float t) { return __float_as_uint(t + 12582912.0f); }

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return prmt(prmt(a, b, 0x0040), prmt(c, d, 0x0040), 0x5410);
}

// v = gamma (v - mean) rstd + beta.
template <int V, int I>
__device__ __forceinline__ void affine(const Span<V, I> &sp, float *v, const Stats &s, const float *gamma,
                                       const float *beta)
{
    float p[V * I];
#pragma unroll
    for (int e = 0; e < V * I; ++e) v[e] = normalised(v[e], s);
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
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __fmaf_rn(normalised(v[e], s), gm[e], bt[e]);
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
    if (!EARLY && (WARP || a.pre == QNN_NORM_NONE || !a.h)) {  // no reduction follows whose barrier would do
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
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __fmaf_rn(normalised(v[e], s), hm[e], hb[e]);
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
    if (sp.t == 0) a.h_scale[row] = __fdiv_rn(m, 127.0f);
    if (m < 0x1p-100f) {  // 127 / m could pass the fp32 range: both sides of h / m times a power of two, exactly
        m *= 0x1p100f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= 0x1p100f;
    }
    const float f = m == 0.0f ? 0.0f : __fdiv_rn(127.0f, m);
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
    __shared__ float slots[2][64];
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
    __shared__ float slots[2][64];
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
        if (!mbar_wait(bar0 + 8 * stage, phase, a.status)) {
            drain_ring(bar0, a.stages, stage, phase, (a.rows - row + step - 1) / step, a.status);
            return;
        }
        const uint8_t *from = ring + (size_t)stage * bytes;
        norm_row<TR, TY, WARP, false>(
            a, sp, row, reinterpret_cast<const TR *>(from), yb ? reinterpret_cast<const TY *>(from + rb) : nullptr,
            gb ? reinterpret_cast<const TY *>(from + rb + yb) : gate_row<TY>(a, row), red, [&] {
                if (sp.t == 0 && row + a.stages * step < a.rows) ask(row + a.stages * step, stage);
            });
        if (++stage == a.stages) stage = 0, phase ^= 1;
    }
}

// ---- launch --------------------------------------------------------------------------

template <typename TR, typename TY, int V, int I, int MAXT>
qnn_status launch_norm(const NormArgs &a, cudaStream_t s)
{
    constexpr int per = V * I;
    if constexpr (MAXT <= 512)
        if (a.C <= 32 * per)
            return launch_dependent(
                block_norm_kernel<TR, TY, V, I, true, per <= 8, 512>, a,
                dim3((unsigned)std::min<int64_t>((a.rows + kWarpRows - 1) / kWarpRows, 16 * sm_count())),
                32 * kWarpRows, 0, s);
    const int threads = (a.C + per * 32 - 1) / (per * 32) * 32;
    return launch_dependent(block_norm_kernel<TR, TY, V, I, false, per <= 8, MAXT>, a,
                            dim3((unsigned)std::min<int64_t>(a.rows, (int64_t)sm_count() * std::max(1024 / threads, 1))), threads, 0, s);
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
    if (!opt_in_smem(kern, kRingSmem, opted_in, kRingCarveout)) return QNN_ERR_CUDA;
    const int64_t want = (a.rows + rows - 1) / rows;
    return launch_dependent(kern, a, dim3((unsigned)std::min<int64_t>(want, (int64_t)sm_count() * blocks)), threads, a.stages * stage, s);
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
    static_assert(3 * kMaxRingC * 4 <= kRingSmem, "a stage of three fp32 rows has to fit");
    const bool many = rows * C >= (int64_t)sm_count() * 16384, ring = many && vec && C <= kMaxRingC;
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
