// qnn_blocknorm_backward.cu -- q_block_norm_backward: the gradients of
//
//   p  = norm_post(y)      r' = a r + b gate p      h = norm_pre(r')
//
// with x^ and y^ the normalised r' and y, and G the gradient at r':
//   G   = dr' + D_pre(gamma_pre dh),   dr = a G,   t = b gate G,   dy = D_post(gamma_post t)
//   D(g) = (g - mean(g) [LAYER only] - x^ mean(g x^)) / sqrt(.)
//   dgate = b sum G p over the rows that share it;   dgamma = sum upstream x^,
//   dbeta = sum upstream   (upstream: dh before, t after)
//
// One pass: a row's r', y, dh and dr' are read once, dr and dy written once, and the
// sums over rows stay in registers.  A block takes a chunk of consecutive rows, one at a
// time, each thread the same columns of every row, so that its column's sums need no
// exchange; at the end of the chunk they go to the workspace, and a second kernel adds
// the blocks' sums in their order.  The statistics are recomputed (two reductions over
// registers) rather than read: the rows are here anyway.  Aligned rows come through a
// ring of stages in shared memory, filled by bulk copies while rows are computed.
#include "qnn_blocknorm.cuh"

namespace qnn {
namespace {

struct BackArgs {
    const void *r, *y, *gate, *dh, *dr_out;  // r: r' as the forward call wrote it
    const float *gamma_post, *beta_post, *gamma_pre;
    void *dr, *dy, *dgate;
    float *ws;       // [block][kSlots][C]
    uint32_t wants;  // bit s: slot s is summed
    int64_t rows, ld_r, ld_y, ld_h, gate_rows, chunk;
    float a, b, eps_post, eps_pre, inv_c;
    int C, post, pre;
    int stages;        // of the ring
    uint32_t *status;  // device status word
};

// A block's sums: the four parameter gradients, and the gate's gradient for a group of
// rows that began in an earlier block's chunk, or that goes on in a later one's.
enum { kGammaPre, kBetaPre, kGammaPost, kBetaPost, kGateHead, kGateTail, kSlots };

// The statistics of two rows of values (r' and y) in the same reductions.
template <int V, int I>
__device__ __forceinline__ void stats_of_two(const Span<V, I> &sp, const float *x, const float *y, bool x_layer,
                                             bool y_layer, const BackArgs &a, RowReduce &red, Stats &sx, Stats &sy)
{
    float2 m = make_float2(0.0f, 0.0f);
    if (x_layer || y_layer) {
#pragma unroll
        for (int e = 0; e < V * I; ++e) m.x += x[e], m.y += y[e];
        m = red.sum<false>(m);
        sx.mean = x_layer ? m.x * a.inv_c : 0.0f;
        sy.mean = y_layer ? m.y * a.inv_c : 0.0f;
    }
    m = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < I; ++i)
        if (sp.in(i))
#pragma unroll
            for (int e = i * V; e < (i + 1) * V; ++e) {
                const float dx = x[e] - sx.mean, dy = y[e] - sy.mean;
                m.x = __fmaf_rn(dx, dx, m.x);
                m.y = __fmaf_rn(dy, dy, m.y);
            }
    m = red.sum<false>(m);
    sx.rstd = rstd_of(m.x, a.inv_c, a.eps_pre);
    sy.rstd = rstd_of(m.y, a.inv_c, a.eps_post);
}

// RING: rows through the ring (V = 8).  REG: sums over rows in registers; rows too wide
// for that (C > 8192) add to the workspace as they go.
template <typename TR, typename TY, int V, int I, bool RING, bool REG, bool BETA>
__global__ void __launch_bounds__(REG ? 512 : 1024)
    block_norm_backward_kernel(const __grid_constant__ BackArgs a)
{
    constexpr int E = V * I;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 slots[2][32];
    __shared__ __align__(8) uint64_t bars[kMaxStages];
    RowReduce red{slots};
    const Span<V, I> sp{(int)threadIdx.x, (int)blockDim.x, a.C};
    const int64_t row0 = blockIdx.x * a.chunk, row1 = min(row0 + a.chunk, a.rows);
    float *part = a.ws + (int64_t)blockIdx.x * kSlots * a.C;
    const bool pre = a.dh && a.pre != QNN_NORM_NONE, post = a.y && a.post != QNN_NORM_NONE;

    // a stage: [r'][y][dh][dr'][gate row], those that every row has
    const int rb = pre ? a.C * (int)sizeof(TR) : 0, yb = a.y ? a.C * (int)sizeof(TY) : 0,
              hb = a.dh ? a.C * (int)sizeof(TY) : 0, ob = a.dr_out ? a.C * (int)sizeof(TR) : 0,
              gb = a.gate && a.gate_rows == 1 ? a.C * (int)sizeof(TY) : 0, bytes = rb + yb + hb + ob + gb;
    const uint32_t bar0 = smem_u32(bars);
    auto ask = [&](int64_t row, int stage) {  // by one thread
        const uint32_t bar = bar0 + 8 * stage;
        uint32_t to = smem_u32(smem + (size_t)stage * bytes);
        mbar_arrive_expect_tx(bar, bytes);
        if (rb) bulk_g2s(to, static_cast<const TR *>(a.r) + row * a.ld_r, rb, bar);
        if (yb) bulk_g2s(to + rb, static_cast<const TY *>(a.y) + row * a.ld_y, yb, bar);
        if (hb) bulk_g2s(to + rb + yb, static_cast<const TY *>(a.dh) + row * a.ld_h, hb, bar);
        to += rb + yb + hb;
        if (ob) bulk_g2s(to, static_cast<const TR *>(a.dr_out) + row * a.ld_r, ob, bar);
        if (gb) bulk_g2s(to + ob, static_cast<const TY *>(a.gate) + row * a.C, gb, bar);
    };
    grid_dependency_launch();
    if constexpr (RING) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < a.stages; ++i) mbar_init(bar0 + 8 * i, 1);
            fence_mbar_init();
            grid_dependency_wait();
            for (int i = 0; i < a.stages && row0 + i < row1; ++i) ask(row0 + i, i);
        }
        __syncthreads();
    }
    grid_dependency_wait();

    float sum[REG ? 4 : 1][REG ? E : 1], gsum[E] = {};  // gsum: the gate's gradient in the current group
    if constexpr (REG) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int e = 0; e < E; ++e) sum[s][e] = 0.0f;
    } else {
        const float zero[E] = {};
        for (int s = 0; s < 4; ++s)
            if (a.wants >> s & 1) sp.store(part + (int64_t)s * a.C, zero);
    }
    // sum[slot] += u w over this thread's vector i
    auto add = [&](int slot, int i, const float *u, const float *w) {
        if (!BETA && !w) return;
        if constexpr (REG) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                sum[slot][i * V + e] = w ? __fmaf_rn(u[e], w[e], sum[slot][i * V + e]) : sum[slot][i * V + e] + u[e];
        } else {
            if (!(a.wants >> slot & 1) || !sp.in(i)) return;
            float *p = part + (int64_t)slot * a.C + sp.col(i), o[V];
            load_v<V>(p, o);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = w ? __fmaf_rn(u[e], w[e], o[e]) : o[e] + u[e];
            store_v<V>(p, o);
        }
    };

    int64_t q = a.gate_rows ? row0 / a.gate_rows : 0;  // the current group, and the row after it
    int64_t q_end = a.gate_rows ? min((q + 1) * a.gate_rows, a.rows) : a.rows;
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t row = row0; row < row1; ++row) {
        const TR *r_row, *o_row;
        const TY *y_row, *h_row, *g_row;
        if constexpr (RING) {
            if (!mbar_wait(bar0 + 8 * stage, phase, a.status)) return;
            const uint8_t *from = smem + (size_t)stage * bytes;
            r_row = reinterpret_cast<const TR *>(from);
            y_row = reinterpret_cast<const TY *>(from + rb);
            h_row = reinterpret_cast<const TY *>(from + rb + yb);
            o_row = reinterpret_cast<const TR *>(from + rb + yb + hb);
            g_row = gb ? reinterpret_cast<const TY *>(from + rb + yb + hb + ob)
                       : static_cast<const TY *>(a.gate) + q * a.C;
        } else {
            r_row = static_cast<const TR *>(a.r) + row * a.ld_r;
            y_row = static_cast<const TY *>(a.y) + row * a.ld_y;
            h_row = static_cast<const TY *>(a.dh) + row * a.ld_h;
            o_row = static_cast<const TR *>(a.dr_out) + row * a.ld_r;
            g_row = static_cast<const TY *>(a.gate) + q * a.C;
        }
        float x[E], g[E];  // r', then x^; dh, then G
        Stats sx{0.0f, 1.0f}, sy{0.0f, 1.0f};
        if (pre) sp.load0(r_row, x);
        else
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.0f;
        if (pre || post) {
            if (post) sp.load0(y_row, g);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 0.0f;
            stats_of_two(sp, x, g, pre && a.pre == QNN_NORM_LAYER, post && a.post == QNN_NORM_LAYER, a, red, sx, sy);
        }
        if (a.dh) sp.load0(h_row, g);
        else
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = 0.0f;
        if (pre) {
            const float c = -sx.mean * sx.rstd;
            float2 m = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float *xv = x + i * V, *gv = g + i * V, gm[V];
                if (a.gamma_pre) load_v<V>(a.gamma_pre + (sp.in(i) ? sp.col(i) : 0), gm);
#pragma unroll
                for (int e = 0; e < V; ++e) xv[e] = __fmaf_rn(xv[e], sx.rstd, c);
                add(kBetaPre, i, gv, nullptr);
                add(kGammaPre, i, gv, xv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (a.gamma_pre) gv[e] *= gm[e];
                    m.x += gv[e];
                    m.y = __fmaf_rn(gv[e], xv[e], m.y);
                }
            }
            m = red.sum<false>(m);
            const float mg = a.pre == QNN_NORM_LAYER ? m.x * a.inv_c : 0.0f, mx = m.y * a.inv_c;
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = sx.rstd * __fmaf_rn(-x[e], mx, g[e] - mg);
        }
        if (a.dr_out) {
            sp.load(o_row, x);
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] += x[e];
        }
        sp.clear(g);  // columns beyond C take no part in the sums to come
        if (a.dr) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = a.a * g[e];
            sp.store(static_cast<TR *>(a.dr) + row * a.ld_r, x);
        }
        if (a.y) {
            sp.load(y_row, x);
            const float c = -sy.mean * sy.rstd;
            float2 m = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int col = sp.in(i) ? sp.col(i) : 0;
                float *xv = x + i * V, *gv = g + i * V, gm[V], w[V], p[V];
                if (a.gamma_post) load_v<V>(a.gamma_post + col, gm);
                if (a.beta_post) load_v<V>(a.beta_post + col, p);
                if (a.gate) load_v<V>(g_row + col, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (post) xv[e] = __fmaf_rn(xv[e], sy.rstd, c);
                    float t = a.gamma_post ? xv[e] * gm[e] : xv[e];
                    if (a.beta_post) t += p[e];
                    gv[e] *= a.b;
                    gsum[i * V + e] = __fmaf_rn(gv[e], t, gsum[i * V + e]);
                    if (a.gate) gv[e] *= w[e];
                }
                add(kBetaPost, i, gv, nullptr);
                add(kGammaPost, i, gv, xv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (a.gamma_post) gv[e] *= gm[e];
                    m.x += gv[e];
                    m.y = __fmaf_rn(gv[e], xv[e], m.y);
                }
            }
            if (post) {
                m = red.sum<false>(m);
                const float mg = a.post == QNN_NORM_LAYER ? m.x * a.inv_c : 0.0f, mx = m.y * a.inv_c;
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = sy.rstd * __fmaf_rn(-x[e], mx, g[e] - mg);
            }
        }
        if constexpr (RING) {
            // all threads have read the stage: behind the last reduction, or a barrier for it
            if (!post) __syncthreads();
            if (threadIdx.x == 0 && row + a.stages < row1) ask(row + a.stages, stage);
            if (++stage == a.stages) stage = 0, phase ^= 1;
        }
        if (a.dy) sp.store(static_cast<TY *>(a.dy) + row * a.ld_y, g);
        if (a.dgate && (row + 1 == q_end || row + 1 == row1)) {
            // the group ends with this row, or the chunk does
            const bool began = q * a.gate_rows >= row0;
            if (began && row + 1 == q_end) sp.store(static_cast<TY *>(a.dgate) + q * a.C, gsum);
            else sp.store(part + (int64_t)(began ? kGateTail : kGateHead) * a.C, gsum);
#pragma unroll
            for (int e = 0; e < E; ++e) gsum[e] = 0.0f;
        }
        if (row + 1 == q_end) {
            ++q;
            q_end = min(q_end + a.gate_rows, a.rows);
        }
    }
    if constexpr (REG) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (a.wants >> s & 1) sp.store(part + (int64_t)s * a.C, sum[s]);
    }
}

struct FinishArgs {
    const float *ws;
    float *out[4];  // dgamma_pre, dbeta_pre, dgamma_post, dbeta_post
    void *dgate;
    int64_t rows, gate_rows, chunk;
    int C, blocks, gate_dt;
    int slot[4], sums;  // the parameter gradients that are wanted
    int by_group;       // the gate's jobs: groups (fewer of them), or boundaries between blocks
};

constexpr int kFinishWarps = 32;

// Adds the blocks' sums in a fixed order.  blockIdx.y: a parameter gradient, then the
// groups of rows that share a gate across blocks, found by their number or by the first
// boundary between two blocks' rows inside them.  32 columns a block, each warp every
// kFinishWarps-th of the sums.
__global__ void __launch_bounds__(kFinishWarps * 32) block_norm_finish_kernel(const __grid_constant__ FinishArgs a)
{
    __shared__ float s[kFinishWarps][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    const bool param = (int)blockIdx.y < a.sums;
    const int job = (int)blockIdx.y - a.sums;
    int b0 = 0, b1 = a.blocks;
    int64_t q = 0;
    grid_dependency_launch();
    if (!param) {
        if (a.by_group) q = job;
        else q = (job + 1) * a.chunk / a.gate_rows;  // the group of the first row behind the boundary
        const int64_t r0 = q * a.gate_rows, r1 = a.gate_rows ? min(r0 + a.gate_rows, a.rows) : a.rows;
        b0 = (int)(r0 / a.chunk);
        b1 = (int)((r1 - 1) / a.chunk) + 1;
        if (b1 - b0 == 1 || (!a.by_group && b0 != job)) return;  // one block's alone, or another boundary's
    }
    grid_dependency_wait();
    float v = 0.0f;
    if (col < a.C)
#pragma unroll 8
        for (int b = b0 + w; b < b1; b += kFinishWarps) {
            const int slot = param ? a.slot[blockIdx.y] : b == b0 ? kGateTail : kGateHead;
            v += a.ws[((int64_t)b * kSlots + slot) * a.C + col];
        }
    s[w][lane] = v;
    __syncthreads();
    if (w != 0 || col >= a.C) return;
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < kFinishWarps; ++k) v += s[k][lane];
    const int64_t at = q * a.C + col;
    if (param) a.out[blockIdx.y][col] = v;
    else if (a.gate_dt == QNN_F32) static_cast<float *>(a.dgate)[at] = v;
    else if (a.gate_dt == QNN_F16) static_cast<__half *>(a.dgate)[at] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16 *>(a.dgate)[at] = from_f32<__nv_bfloat16>(v);
}

// ---- launch --------------------------------------------------------------------------

#ifndef EIGHT
#define EIGHT 4096
#endif
#ifndef THR8
#define THR8 512
#endif
// Threads that hold a row: 8 columns each up to 2048, 16 up to 8192, 32 beyond.
int back_threads(int C)
{
    const int per = 32 * (C <= EIGHT ? 8 : C <= 8192 ? 16 : 32);
    return (C + per - 1) / per * 32;
}

// Blocks that an SM's registers hold (about 80, 128 and 64 a thread), 8 at most: more
// blocks are more sums to add.
int back_blocks_per_sm(int C)
{
    const int threads = C <= EIGHT ? THR8 : C <= 8192 ? 512 : 1024;
    return std::max(1, std::min(8, threads / back_threads(C)));
}

struct BackPlan {
    int64_t chunk;  // rows of a block
    int blocks, stages;
};

BackPlan back_plan(int64_t rows, int C, int stage)
{
    BackPlan p;
    int per_sm = back_blocks_per_sm(C);
    // two stages for each block where that leaves half the blocks or more
    p.stages = 1;
    if (stage > 0) {
        if (kRingSmem / (2 * stage) >= std::max(1, per_sm / 2)) per_sm = std::min(per_sm, kRingSmem / (2 * stage));
        else per_sm = std::max(1, std::min(per_sm, kRingSmem / stage));
        p.stages = std::max(1, std::min(kMaxStages, kRingSmem / (per_sm * stage)));
    }
    const int64_t most = (int64_t)sm_count() * per_sm;
    p.chunk = std::max<int64_t>(1, (rows + most - 1) / most);
    p.blocks = (int)((rows + p.chunk - 1) / p.chunk);
    return p;
}

template <typename TR, typename TY, int V, int I, bool RING, bool REG, bool BETA>
qnn_status launch_back(BackArgs a, const BackPlan &p, int stage, cudaStream_t s)
{
    auto kern = block_norm_backward_kernel<TR, TY, V, I, RING, REG, BETA>;
    a.stages = p.stages;
    if (RING) {
        static std::atomic<uint64_t> opted_in{0};
        if (!opt_in_smem(kern, kMaxRing, opted_in, kRingCarveout)) return QNN_ERR_CUDA;
    }
    return launch_dependent(kern, a, p.blocks, back_threads(a.C), RING ? p.stages * stage : 0, s);
}

}  // namespace
}  // namespace qnn

extern "C" size_t qnn_block_norm_backward_workspace_bytes(int64_t rows, int C, const qnn_block_norm *p)
{
    using namespace qnn;
    if (!p || rows < 0 || C <= 0 || C > kMaxC) return 0;
    // the most blocks that any types lead to
    return (size_t)std::min<int64_t>(rows, (int64_t)sm_count() * back_blocks_per_sm(C)) * kSlots * C * sizeof(float);
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
    a.rows = rows, a.gate_rows = p->gate_rows, a.C = C, a.post = p->post, a.pre = p->pre;
    a.ld_r = p->ld_r ? p->ld_r : C, a.ld_y = p->ld_y ? p->ld_y : C, a.ld_h = p->ld_h ? p->ld_h : C;
    a.a = p->res_scale, a.b = p->block_scale, a.eps_post = p->eps_post, a.eps_pre = p->eps_pre, a.inv_c = 1.0f / C;
    a.wants = (dgamma_pre ? 1u << kGammaPre : 0) | (dbeta_pre ? 1u << kBetaPre : 0) |
              (dgamma_post ? 1u << kGammaPost : 0) | (dbeta_post ? 1u << kBetaPost : 0);
    a.status = status_word();
    if (!a.status) return QNN_ERR_CUDA;
    const int er = float_bytes(r_dt), ey = float_bytes(y_dt);
    const bool vec = C % 8 == 0 && rows_aligned(a.ld_r, er) && (!y || rows_aligned(a.ld_y, ey)) &&
                     (!dh || rows_aligned(a.ld_h, ey));
    const int stage = C * ((dh && p->pre != QNN_NORM_NONE ? er : 0) + (y ? ey : 0) + (dh ? ey : 0) + (dr_out ? er : 0) +
                           (p->gate && p->gate_rows == 1 ? ey : 0));
    const bool ring = vec && C <= 8192 && stage <= kMaxRing;
    const bool beta = dbeta_pre || dbeta_post;
    const BackPlan plan = back_plan(rows, C, ring ? stage : 0);
    a.chunk = plan.chunk;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows > 0) {
        qnn_status done = QNN_OK;
        with_types(r_dt, y_dt, [&](auto tr, auto ty) {
            using TR = decltype(tr);
            using TY = decltype(ty);
            if (ring && C <= EIGHT) done = beta ? launch_back<TR, TY, 8, 1, true, true, true>(a, plan, stage, s) : launch_back<TR, TY, 8, 1, true, true, false>(a, plan, stage, s);
            else if (ring) done = beta ? launch_back<TR, TY, 8, 2, true, true, true>(a, plan, stage, s) : launch_back<TR, TY, 8, 2, true, true, false>(a, plan, stage, s);
            else if (C <= EIGHT) done = launch_back<TR, TY, 1, 8, false, true, true>(a, plan, 0, s);
            else if (C <= 8192) done = launch_back<TR, TY, 1, 16, false, true, true>(a, plan, 0, s);
            else if (vec) done = launch_back<TR, TY, 8, 4, false, false, true>(a, plan, 0, s);
            else done = launch_back<TR, TY, 1, 32, false, false, true>(a, plan, 0, s);
        });
        if (done != QNN_OK || !sums) return done;
    }
    if (!sums) return QNN_OK;
    if (rows == 0 && dgate && !p->gate_rows && cudaMemsetAsync(dgate, 0, (size_t)C * ey, s) != cudaSuccess) {
        (void)cudaGetLastError();
        return QNN_ERR_CUDA;
    }
    FinishArgs f{};
    f.ws = a.ws;
    float *const out[4] = {dgamma_pre, dbeta_pre, dgamma_post, dbeta_post};
    for (int i = 0; i < 4; ++i)
        if (out[i]) f.slot[f.sums] = i, f.out[f.sums++] = out[i];
    f.dgate = dgate, f.gate_dt = y_dt, f.rows = rows, f.gate_rows = p->gate_rows, f.chunk = a.chunk, f.C = C;
    f.blocks = plan.blocks;
    int64_t jobs = 0;
    if (dgate && f.blocks > 1) {
        const int64_t groups = p->gate_rows ? (rows + p->gate_rows - 1) / p->gate_rows : 1;
        f.by_group = groups < f.blocks;
        jobs = p->gate_rows == 1 ? 0 : f.by_group ? groups : f.blocks - 1;
    }
    const dim3 grid((C + 31) / 32, (unsigned)(f.sums + jobs));
    if (grid.y == 0) return QNN_OK;
    return launch_dependent(block_norm_finish_kernel, f, grid, kFinishWarps * 32, 0, s);
}
