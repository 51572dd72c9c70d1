// qnn_gemv_columns.cu -- qgemv_w4 for more rows of x than one mma.sync tile holds: the
// same weights image, up to 32 columns of x on the 5th-generation tensor cores.
//
// With 32 columns an mma.sync kernel reads every fragment of x from shared memory once
// for each 16 or 32 channels, and is bound by that.  Here a block has 128 channels as
// the M of tcgen05.mma: the codes go as f16 / bf16 integers to tensor memory as the A
// operand (they never touch shared memory), x is read from shared memory by the MMA
// itself, once for 128 channels, and the sums of a scale's group come out of tensor
// memory to be scaled and added in fp32 registers.
//
// Roles of a block's warps, one step of 128 input channels at a time:
//   16      codes of 16 channels, every other step: global -> registers -> A
//   4 or 8  sums: 32 channels by 16 columns of D -> registers, times the scale, added
//   4       x: every fourth step each, global -> shared memory as it is -> B
//   2       MMA: one thread each, every other step (a step's D is its own, so the two
//           need no order; one thread alone took 1100 cycles a step, most of it waits)
// A and B have four stages, D up to four slots.  Two mbarriers a stage: `full` (its codes
// and x are there, its D slot has been read) and `done` (its MMAs are).  The fragment
// layout of the image is that of tcgen05.st's 16 x 128 bit shape, so a lane's registers
// are stored as they come: word f of a lane makes columns 8 f .. 8 f + 7 of the step's 64
// (two f16 a column), and x is put down in the order of K that this gives.
//
// Measured: 32 rows, 16384 x 4096, bf16, groups of 128: 20.0 us over weights that L2 cannot
// hold (1.8 TB/s, 0.27 of a copy's bandwidth), 17.6 over three copies in turn (mma.sync forms
// took 33 and 37 there), about 800 cycles a step where its 8 KB at 23 bytes a clock would
// take 350.  Issuing half the MMAs changed nothing, so it is
// the latency of the hand-overs between the roles and not the tensor core that bounds it.
#include <cooperative_groups.h>
#include <type_traits>
#include "qnn_gemv.cuh"

namespace qnn {
namespace {

namespace cg = cooperative_groups;

constexpr int kTiles = 8, kCodeWarps = 2 * kTiles, kXWarps = 4, kMmaWarps = 2, kStages = 4;
// four warps (the quadrants of tensor memory) for each 16 columns of sums
template <int NC>
constexpr int kSumWarps = NC / 4;
template <int NC>
constexpr int kThreads = (kCodeWarps + kSumWarps<NC> + kXWarps + kMmaWarps) * 32;
constexpr uint32_t kTmemCols = 512, kDCol = 256;  // A: 4 stages of 64 columns, then D

// A from tensor memory, B from shared memory, fp32 D.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 lanes x 64 columns: register 2 i + h of lane 4 g + j is row g + 8 h, column 4 i + j.
__device__ __forceinline__ void tmem_st_16x128b_x16(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// A unit: 32 values of a row of x, 16-byte chunks of them 512 bytes apart (a lane's units
// then meet no bank conflict).  Asked for by asynchronous copies; zero beyond K.
template <int XT>
constexpr int kUnitChunks = XT == QNN_F32 ? 8 : 4;

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from, int valid)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(valid)
                 : "memory");
}

template <int XT>
__device__ __forceinline__ void ask_unit(const GemvArgs &a, int64_t row, int k, uint32_t to)
{
    constexpr int ES = XT == QNN_F32 ? 4 : 2;
    const uint8_t *p = static_cast<const uint8_t *>(a.x) + row * a.ldx * ES;  // of the row; K's end is inside it
    const int64_t first = (int64_t)k * ES, end = (int64_t)a.K * ES;
    auto copies = [&](auto width) {
        constexpr int B = decltype(width)::value;
#pragma unroll
        for (int c = 0; c < kUnitChunks<XT>; ++c)
#pragma unroll
            for (int b = 0; b < 16; b += B) {
                const int64_t at = first + 16 * c + b;
                const int valid = (int)min(max(end - at, (int64_t)0), (int64_t)B);
                copy_async<B>(to + 512 * c + b, p + (valid ? at : 0), valid);
            }
    };
    if (a.align == 16) copies(std::integral_constant<int, 16>{});
    else if (a.align == 8) copies(std::integral_constant<int, 8>{});
    else if (XT == QNN_F32 || a.align == 4) copies(std::integral_constant<int, 4>{});
    else
        for (int i = 0; i < 16; ++i) {  // rows on odd 16-bit addresses
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p) + k + 2 * i;
            const uint32_t lo = k + 2 * i < a.K ? load_input(q) : 0, hi = k + 2 * i + 1 < a.K ? load_input(q + 1) : 0;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 512 * (i / 4) + 4 * (i % 4)), "r"(lo | hi << 16) : "memory");
        }
}

// ... to the stage's B operand: rows (columns of x) of 64 channels, 128 bytes, 128-byte
// swizzled, two such halves a stage; channels part * 32 .. + 31.
template <int XT, int NC>
__device__ __forceinline__ void put_unit(uint32_t stage, int tok, int part, uint32_t from)
{
    constexpr int P = Cols<XT>::kParts;
    uint32_t w[4 * kUnitChunks<XT>];
#pragma unroll
    for (int c = 0; c < kUnitChunks<XT>; ++c) {
        const uint4 u = lds_v4(from + 512 * c);
        w[4 * c] = u.x, w[4 * c + 1] = u.y, w[4 * c + 2] = u.z, w[4 * c + 3] = u.w;
    }
    const uint32_t half = stage + (uint32_t)(part >> 1) * (NC * 128);
    auto put = [&](int row, int q, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
        const int chunk = 4 * (part & 1) + q;
        sts_v4(half + row * 128 + ((chunk ^ (row & 7)) << 4), w0, w1, w2, w3);
    };
    if constexpr (XT != QNN_F32) {
#pragma unroll
        for (int q = 0; q < 4; ++q) put(tok, q, w[q], w[4 + q], w[8 + q], w[12 + q]);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t o[P][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t lo[3], hi[3];
                bf16_parts(__uint_as_float(w[8 * j + 2 * q]), lo);
                bf16_parts(__uint_as_float(w[8 * j + 2 * q + 1]), hi);
#pragma unroll
                for (int p = 0; p < P; ++p) o[p][j] = lo[p] | hi[p] << 16;
            }
#pragma unroll
            for (int p = 0; p < P; ++p) put(tok * P + p, q, o[p][0], o[p][1], o[p][2], o[p][3]);
        }
    }
}

// NC: columns of x, a multiple of 16.  NS: scales in a step.
template <int XT, int NC, bool ZERO, int NS>
__global__ void __launch_bounds__(kThreads<NC>, 1) gemv_w4_columns_kernel(const __grid_constant__ GemvArgs a)
{
    constexpr bool BF16 = XT != QNN_F16;
    constexpr int P = Cols<XT>::kParts, TOK = NC / P, PITCH = NC + 1;
    constexpr int kXWarp0 = kCodeWarps + kSumWarps<NC>, kMmaWarp0 = kXWarp0 + kXWarps;
    constexpr uint32_t STAGE = NC * 256, SLOT = NS * NC;  // bytes of B, columns of D
    constexpr int SLOTS = 256 / SLOT < kStages ? 256 / SLOT : kStages;
    extern __shared__ __align__(16) uint8_t raw[];
    uint8_t *smem = raw + (-smem_u32(raw) & 1023u);  // the swizzle's atoms
    __shared__ __align__(8) uint64_t bars[2][kStages], end_bars[kMmaWarps];
    __shared__ uint32_t tmem_slot;
    // a stage's x as it comes: units of the block's rows, 32 of them at a time
    constexpr uint32_t RAW = (TOK * 4 + 31) / 32 * 512 * kUnitChunks<XT>;
    uint8_t *raw_x = smem + kStages * STAGE;
    float *part = reinterpret_cast<float *>(raw_x + kStages * RAW);  // [128][PITCH]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t m0 = (int64_t)blockIdx.y * TOK;
    const int toks = (int)min((int64_t)TOK, a.M - m0);
    const int splits = gridDim.z, rank = blockIdx.z;
    const int b0 = a.steps * rank / splits, n = a.steps * (rank + 1) / splits - b0;
    const uint32_t full = smem_u32(bars[0]), done = smem_u32(bars[1]);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, kTiles + 1 + kSumWarps<NC>);
            mbar_init(done + 8 * i, 1);
        }
        for (int i = 0; i < kMmaWarps; ++i) mbar_init(smem_u32(&end_bars[i]), 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp0) {
        tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // only now: a block of the next grid that took tensor memory first and waited for
    // this grid would keep it from blocks of this one
    grid_dependency_launch();

    bool ok = true;
    auto wait = [&](uint32_t bar, int use) {  // the use-th phase of a barrier, by a whole warp
        ok = __all_sync(0xffffffffu, mbar_wait_idle(bar, (uint32_t)use & 1u, a.status));
        return ok;
    };
    if (warp < kCodeWarps) {
        // lanes 32 (w % 4) + 16 (w / 4 % 2) .. + 15 of tensor memory, steps w / 8, + 2, ...
        const int row16 = 2 * (warp & 3) + (warp >> 2 & 1), odd = warp >> 3;
        const int64_t tile = min((int)blockIdx.x * 8 + row16, a.tiles - 1);  // beyond N: computed, not stored
        const uint32_t at = tmem + ((uint32_t)(row16 * 16) << 16);
        const uint8_t *wp = a.w + (tile * a.steps + b0) * 1024;
        if (lane == 0 && n > 0 && !odd) prefetch_l2(wp, min(n, 64) * 1024);  // the rest of a long run would only crowd L2
        wp += odd * 1024 + lane * 32;
        grid_dependency_wait();
        const uint8_t *zp = ZERO ? a.zero + tile * a.groups * 16 + (lane >> 2) * 2 : nullptr;
        constexpr int U = 2;
        uint32_t w[U][8], z[U][NS];
        auto fetch = [&](int u, int t) {
            ldg_stream_v8(wp, w[u]);
            wp += 2048;
#pragma unroll
            for (int q = 0; q < NS; ++q) {
                if constexpr (ZERO) {
                    const int g = (uint32_t)((b0 + t) * NS + q) / (uint32_t)a.per_scale;
                    z[u][q] = load_input(reinterpret_cast<const uint16_t *>(zp + (int64_t)min(g, a.groups - 1) * 16));
                } else {
                    z[u][q] = 0x0808u;
                }
            }
        };
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (odd + 2 * u < n) fetch(u, odd + 2 * u);
        for (int t0 = odd; t0 < n && ok; t0 += 2 * U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + 2 * u, stage = t % kStages;
                if (t >= n) break;
                uint32_t r[32];
#pragma unroll
                for (int f = 0; f < 8; ++f) {
                    const uint32_t zz = z[u][f * NS / 8];
                    uint32_t o[4];
                    codes_to_a<BF16>(w[u][f], zero_term<BF16>(zz & 0xffu, zz >> 8), o);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[4 * f + e] = o[e];
                }
                if (t + 2 * U < n) fetch(u, t + 2 * U);
                if (!wait(done + 8 * stage, t / kStages + 1)) break;  // the MMAs four steps ago
                tc_fence_after();
                tmem_st_16x128b_x16(at + 64 * stage, r);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * stage);
            }
        }
    } else if (warp < kXWarp0) {
        const int q = warp & 3, ch = q * 32 + lane, r = ch & 15, col0 = (warp - kCodeWarps) / 4 * 16;
        const int64_t tile = min((int)blockIdx.x * 8 + ch / 16, a.tiles - 1);
        const int64_t at = tile * a.groups * 16 + (r & 7) * 2 + (r >> 3);
        float sum[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[c] = 0.0f;
        int gn = (uint32_t)(b0 * NS) / (uint32_t)a.per_scale, left = a.per_scale - (b0 * NS - gn * a.per_scale);
        grid_dependency_wait();
        // the scales of steps to come, a wait for memory ahead
        constexpr int A = 8;
        uint32_t ahead[A];
        auto next_scale = [&]() {
            const uint32_t v = load_scale(a.scale, a.scale_dt, at + (int64_t)min(gn, a.groups - 1) * 16);
            if (--left == 0) left = a.per_scale, ++gn;
            return v;
        };
#pragma unroll
        for (int i = 0; i < A; ++i) ahead[i] = next_scale();
        if (lane == 0)
            for (int t = 0; t < SLOTS; ++t) mbar_arrive(full + 8 * t);  // the slots are free
        for (int t0 = 0; t0 < n && ok; t0 += A / NS) {
#pragma unroll
            for (int i = 0; i < A; i += NS) {
                const int t = t0 + i / NS, stage = t % kStages;
                if (t >= n) break;
                if (!wait(done + 8 * stage, t / kStages)) break;
                tc_fence_after();
                const uint32_t from = tmem + ((uint32_t)(q * 32) << 16) + kDCol + SLOT * (t % SLOTS);
#pragma unroll
                for (int sub = 0; sub < NS; ++sub) {
                    const float s = scale_f32(ahead[i + sub], a.scale_dt);
                    ahead[i + sub] = next_scale();
                    uint32_t v[16];
                    tmem_ld16(from + sub * NC + col0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 16; ++c) sum[c] = __fmaf_rn(__uint_as_float(v[c]), s, sum[c]);
                }
                tc_fence_before();
                __syncwarp();
                // the slot's next step may go on; its barrier's last phase is over, as this step is
                if (lane == 0 && t + SLOTS < n) mbar_arrive(full + 8 * ((t + SLOTS) % kStages));
            }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) part[ch * PITCH + col0 + c] = sum[c];
    } else if (warp < kMmaWarp0) {
        // unit u of a step: row u / 4 of the block's, channels 32 (u % 4) .. + 31; a lane's are
        // lane, lane + 32, ...: the same channels of every eighth row
        constexpr int UNITS = (TOK * 4 + 31) / 32, UB = 512 * kUnitChunks<XT>, ES = XT == QNN_F32 ? 4 : 2;
        const int first = warp - kXWarp0, units = toks * 4, tok = lane >> 2, quarter = lane & 3;
        const uint32_t stage = smem_u32(smem) + first * STAGE, raw0 = smem_u32(raw_x) + first * RAW + lane * 16;
        const uint8_t *from = static_cast<const uint8_t *>(a.x) + ((m0 + tok) * a.ldx + quarter * 32) * ES;
        const int64_t eight_rows = 8 * a.ldx * ES;
        auto ask = [&](int t) {
            const int k = (b0 + t) * 128;
            if (a.align == 16 && k + 128 <= a.K) {
#pragma unroll
                for (int i = 0; i < UNITS; ++i)
                    if (lane + 32 * i < units) {
                        const uint8_t *p = from + i * eight_rows + (int64_t)k * ES;
#pragma unroll
                        for (int c = 0; c < kUnitChunks<XT>; ++c) copy_async<16>(raw0 + i * UB + 512 * c, p + 16 * c, 16);
                    }
            } else {
                for (int i = 0; i < UNITS; ++i)
                    if (lane + 32 * i < units)
                        ask_unit<XT>(a, m0 + tok + 8 * i, k + quarter * 32, raw0 + i * UB);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        grid_dependency_wait();
        if (first < n) ask(first);
        for (int t = first; t < n; t += kStages) {
            if (!wait(done + 8 * first, t / kStages + 1)) break;
            asm volatile("cp.async.wait_group 0;" ::: "memory");  // a lane reads only what it asked for
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                if (lane + 32 * i < units) put_unit<XT, NC>(stage, tok + 8 * i, quarter, raw0 + i * UB);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full + 8 * first);
            if (t + kStages < n) ask(t + kStages);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");  // none in flight, after a wait that gave up either
    } else {
        // the grid before reads and writes nothing of this role's: so that its time is not taken
        // by polls, nor counted by their limit
        grid_dependency_wait();
        if (lane == 0 && warp < kMmaWarp0 + kMmaWarps) {
            // a serial bottleneck: all that an MMA needs is a constant away from a few
            // registers (descriptor addresses count 16 bytes)
            constexpr uint32_t idesc = idesc_f32acc(BF16 ? 1 : 0, BF16 ? 1 : 0, 128, NC);
            const uint64_t b_desc0 = sdesc_sw128(smem_u32(smem));
            for (int t = warp - kMmaWarp0; t < n; t += kMmaWarps) {
                const int stage = t % kStages;
                const uint32_t a_cols = tmem + 64 * stage, d_cols = tmem + kDCol + SLOT * (t % SLOTS);
                const uint64_t b_desc = b_desc0 + (uint64_t)(stage * (STAGE >> 4));
                if (!mbar_wait(full + 8 * stage, (uint32_t)(t / kStages) & 1u, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int f = 0; f < 8; ++f)
                    mma_f16_ts(d_cols + (f * NS / 8) * NC, a_cols + 8 * f,
                               b_desc + (f >> 2) * (NC * 128 >> 4) + (f & 3) * 2, idesc, f % (8 / NS) > 0);
                mma_commit(done + 8 * stage);
            }
            // nothing of this thread's is in flight when the block ends
            const uint32_t end = smem_u32(&end_bars[warp - kMmaWarp0]);
            mma_commit(end);
            (void)mbar_wait(end, 0, a.status);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp0) tmem_dealloc(tmem, kTmemCols);
    if (splits > 1) cg::this_cluster().sync();
    // 128 channels of one row of x at a time, by the warps that converted the codes
    if (warp < kCodeWarps) {
        const int ch = threadIdx.x & 127;
        const int64_t nn = (int64_t)blockIdx.x * 128 + ch;
        const float bias = a.bias && nn < a.N ? load_input(a.bias + nn) : 0.0f;
        for (int tok = (threadIdx.x >> 7) + 4 * rank; tok < toks && nn < a.N; tok += 4 * splits) {
            float v = 0.0f;
            for (int q = 0; q < splits; ++q) {
                const float *from =
                    (splits > 1 ? cg::this_cluster().map_shared_rank(part, q) : part) + ch * PITCH + tok * P;
#pragma unroll
                for (int p = P - 1; p >= 0; --p) v = __fadd_rn(v, from[p]);  // the small parts first
            }
            if (a.bias) v = __fadd_rn(v, bias);
            store_y(a, (m0 + tok) * a.ldy + nn, v);
        }
    }
    if (splits > 1) cg::this_cluster().sync();  // no block leaves while its sums are read
}

template <int XT, int NC, bool ZERO, int NS>
qnn_status launch(const GemvArgs &a, cudaStream_t s)
{
    constexpr int TOK = NC / Cols<XT>::kParts;
    const int64_t by = (a.M + TOK - 1) / TOK, bx = (a.tiles + 7) / 8;
    // K split over a cluster while the blocks still run all at once and keep two steps each
    int splits = 1;
    while (splits < 4 && bx * by * splits * 2 <= sm_count() && a.steps >= 4 * splits) splits *= 2;
    // One block on an SM, whatever it needs: two could each hold the tensor memory that the
    // other's cluster waits for.
    constexpr int NEED = 1024 + kStages * (NC * 256 + (TOK * 4 + 31) / 32 * 512 * kUnitChunks<XT>) + 128 * (NC + 1) * 4,
                  SMEM = NEED > (120 << 10) ? NEED : 120 << 10;
    auto kern = gemv_w4_columns_kernel<XT, NC, ZERO, NS>;
    static std::atomic<uint64_t> opted_in{0};
    if (!opt_in_smem(kern, SMEM, opted_in)) return QNN_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)bx, (unsigned)by, (unsigned)splits);
    cfg.blockDim = dim3(kThreads<NC>);
    cfg.dynamicSmemBytes = SMEM;
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

template <int XT, int NC, bool ZERO>
qnn_status launch_group(GemvArgs a, int group, cudaStream_t s)
{
    a.per_scale = group % 128 == 0 ? group / 128 : group % 64 == 0 ? group / 64 : group / 32;
    if (group % 128 == 0) return launch<XT, NC, ZERO, 1>(a, s);
    if (group % 64 == 0) return launch<XT, NC, ZERO, 2>(a, s);
    return launch<XT, NC, ZERO, 4>(a, s);
}

template <int XT>
qnn_status launch_type(const GemvArgs &a, int group, cudaStream_t s)
{
    const int64_t cols = a.M * Cols<XT>::kParts;
    if (cols <= 16) return a.zero ? launch_group<XT, 16, true>(a, group, s) : launch_group<XT, 16, false>(a, group, s);
    return a.zero ? launch_group<XT, kMaxCols, true>(a, group, s) : launch_group<XT, kMaxCols, false>(a, group, s);
}

}  // namespace

qnn_status launch_gemv_columns(const GemvArgs &a, int x_dt, int group, cudaStream_t s)
{
    switch (x_dt) {
    case QNN_F32: return launch_type<QNN_F32>(a, group, s);
    case QNN_F16: return launch_type<QNN_F16>(a, group, s);
    default: return launch_type<QNN_BF16>(a, group, s);
    }
}

}  // namespace qnn
