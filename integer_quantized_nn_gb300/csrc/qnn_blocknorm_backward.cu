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
// registers) rather than read: the rows are here anyway.  Rows come through a ring of
// stages in shared memory, filled by bulk copies while rows are computed.
//
// Measured, over data that L2 cannot hold: 4096 x 4096 bf16, RMS norms, one gate: 59 us, 3.4
// TB/s (0.50 of a copy's bandwidth); 12608 x 1024 fp32, LAYER norms with betas: 80 us, 3.9
// TB/s; 8192 x 2003 bf16 104 us (158 without the ring, which cost 4096 x 4096 1 us); 65 x 1003
// 12.0 us (9.6 out of L2).  At 4096 x 4096 no unit is at its limit: 58 instructions an
// element, issue 50 %, 15 warps an SM (128 registers), the stalls spread over fixed latencies,
// shared memory, global loads and barriers.  Beyond 8192 columns a thread holds 32 of them in
// 64 registers and spills (by the compiler's count 7 KB a thread, 4 KB at odd widths): 2048 x
// 16384 bf16 766 us, 0.5 TB/s, with LAYER norms 787; 2048 x 16385 1034 us.
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
    int64_t ring_rows; // the rows that come through it
    uint32_t *status;  // device status word
};

// A block's sums: the four parameter gradients, and the gate's gradient for a group of
// rows that began in an earlier block's chunk, or that goes on in a later one's.
enum { kGammaPre, kBetaPre, kGammaPost, kBetaPost, kGateHead, kGateTail, kSlots };

// A thread's columns as pairs of fp32, for two operations in one instruction: vectors t,
// t + threads, ... of V = 8 columns, four pairs each (a "group"), or single columns, two
// of them a pair and a group.  Loads read column 0 in place of one beyond C; sums leave
// those groups out (keep).
template <int V, int I>
struct PairSpan {
    static constexpr int N = V * I / 2, GP = V == 8 ? 4 : 1, G = N / GP;  // pairs, pairs of a group, groups
    int t, threads, C;
    __device__ __forceinline__ int col(int i) const { return (t + i * threads) * V; }
    __device__ __forceinline__ bool in(int i) const { return col(i) < C; }
    template <typename T>
    __device__ __forceinline__ void load_group(const T *row, int g, float2 *v) const
    {
        if constexpr (V == 8) {
            load_v<8>(row + (in(g) ? col(g) : 0), reinterpret_cast<float *>(v));
        } else {
            v[0].x = to_f32(row[in(2 * g) ? col(2 * g) : 0]);
            v[0].y = to_f32(row[in(2 * g + 1) ? col(2 * g + 1) : 0]);
        }
    }
    template <typename T>
    __device__ __forceinline__ void store_group(T *row, int g, const float2 *v) const
    {
        if constexpr (V == 8) {
            if (in(g)) store_v<8>(row + col(g), reinterpret_cast<const float *>(v));
        } else {
            if (in(2 * g)) row[col(2 * g)] = from_f32<T>(v[0].x);
            if (in(2 * g + 1)) row[col(2 * g + 1)] = from_f32<T>(v[0].y);
        }
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, float2 *v) const
    {
#pragma unroll
        for (int g = 0; g < G; ++g) load_group(row, g, v + g * GP);
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, const float2 *v) const
    {
#pragma unroll
        for (int g = 0; g < G; ++g) store_group(row, g, v + g * GP);
    }
    // the sum with group g's part where that is inside the row, without it elsewhere
    __device__ __forceinline__ float2 keep(int g, float2 with, float2 without) const
    {
        const bool a = V == 8 ? in(g) : in(2 * g), b = V == 8 ? a : in(2 * g + 1);
        return make_float2(a ? with.x : without.x, b ? with.y : without.y);
    }
};

__device__ __forceinline__ float across(float2 v) { return v.x + v.y; }

// The statistics of two rows of values (r' and y) in the same reductions.
template <bool LAYER, int V, int I>
__device__ __forceinline__ void stats_of_two(const PairSpan<V, I> &sp, const float2 *x, const float2 *y,
                                             const BackArgs &a, RowReduce &red, Stats &sx, Stats &sy)
{
    using S = PairSpan<V, I>;
    float2 sum_x = both(0.0f), sum_y = both(0.0f);
    if (LAYER) {
#pragma unroll
        for (int g = 0; g < S::G; ++g) {
            float2 tx = sum_x, ty = sum_y;
#pragma unroll
            for (int k = g * S::GP; k < (g + 1) * S::GP; ++k) tx = add2(tx, x[k]), ty = add2(ty, y[k]);
            sum_x = sp.keep(g, tx, sum_x);
            sum_y = sp.keep(g, ty, sum_y);
        }
        const float2 m = red.sum<false>(make_float2(across(sum_x), across(sum_y)));
        sx.mean = a.pre == QNN_NORM_LAYER ? mean_of(m.x, a.C, a.inv_c) : 0.0f;
        sy.mean = a.post == QNN_NORM_LAYER ? mean_of(m.y, a.C, a.inv_c) : 0.0f;
        sum_x = sum_y = both(0.0f);
    }
    const float2 mx = both(-sx.mean), my = both(-sy.mean);
#pragma unroll
    for (int g = 0; g < S::G; ++g) {
        float2 tx = sum_x, ty = sum_y;
#pragma unroll
        for (int k = g * S::GP; k < (g + 1) * S::GP; ++k) {
            const float2 dx = LAYER ? add2(x[k], mx) : x[k], dy = LAYER ? add2(y[k], my) : y[k];
            tx = fma2(dx, dx, tx);
            ty = fma2(dy, dy, ty);
        }
        sum_x = sp.keep(g, tx, sum_x);
        sum_y = sp.keep(g, ty, sum_y);
    }
    const float2 m = red.sum<false>(make_float2(across(sum_x), across(sum_y)));
    sx.rstd = rstd_of(m.x, a.inv_c, a.eps_pre);
    sy.rstd = rstd_of(m.y, a.inv_c, a.eps_post);
}

// g = (g - mean(g) [LAYER] - x mean(g x)) rstd, from a thread's parts of the sums.
template <bool LAYER, int V, int I>
__device__ __forceinline__ void gradient(const PairSpan<V, I> &, float2 *g, const float2 *x, float2 sg, float2 sgx,
                                         bool layer, float rstd, float inv_c, RowReduce &red)
{
    const float2 rs = both(rstd);
    if (LAYER) {
        const float2 m = red.sum<false>(make_float2(across(sg), across(sgx)));
        const float2 mg = both(layer ? -m.x * inv_c : 0.0f), mx = both(-m.y * inv_c);
#pragma unroll
        for (int k = 0; k < V * I / 2; ++k) g[k] = mul2(rs, fma2(x[k], mx, add2(g[k], mg)));
    } else {
        const float2 mx = both(-red.sum<false>(across(sgx)) * inv_c);
#pragma unroll
        for (int k = 0; k < V * I / 2; ++k) g[k] = mul2(rs, fma2(x[k], mx, g[k]));
    }
}

// RING: rows through the ring.  FULL: a LAYER norm or a beta takes part; without
// them half the sums over rows are not there.
template <typename TR, typename TY, int V, int I, bool RING, bool FULL>
__global__ void __launch_bounds__(V * I <= 16 ? 512 : 1024, 1)
    block_norm_backward_kernel(const __grid_constant__ BackArgs a)
{
    using S = PairSpan<V, I>;
    constexpr int N = S::N, GP = S::GP;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float slots[2][64];
    __shared__ __align__(8) uint64_t bars[kMaxStages];
    RowReduce red{slots};
    const S sp{(int)threadIdx.x, (int)blockDim.x, a.C};
    const int64_t row0 = blockIdx.x * a.chunk, row1 = min(row0 + a.chunk, a.rows);
    float *part = a.ws + (int64_t)blockIdx.x * kSlots * a.C;
    const bool pre = a.dh && a.pre != QNN_NORM_NONE, post = a.y && a.post != QNN_NORM_NONE;

    // a stage: [r'][y][dh][dr'][gate row], those that every row has
    const bool own_gate = a.gate && a.gate_rows == 1;
    const int rr = window_room<V>(a.C, sizeof(TR)), yr = window_room<V>(a.C, sizeof(TY));
    const int rb = pre ? rr : 0, yb = a.y ? yr : 0, hb = a.dh ? yr : 0, ob = a.dr_out ? rr : 0, gb = own_gate ? yr : 0,
              bytes = rb + yb + hb + ob + gb;
    const uint32_t bar0 = smem_u32(bars);
    auto ask = [&](int64_t row, int stage) {  // by one thread
        if (V == 1 && row >= a.ring_rows) return;
        const uint32_t bar = bar0 + 8 * stage;
        uint32_t to = smem_u32(smem + (size_t)stage * bytes);
        const Window r = window<V, TR>(a.r, row, a.ld_r, a.C), y = window<V, TY>(a.y, row, a.ld_y, a.C),
                     h = window<V, TY>(a.dh, row, a.ld_h, a.C), o = window<V, TR>(a.dr_out, row, a.ld_r, a.C),
                     g = window<V, TY>(a.gate, row, a.C, a.C);
        mbar_arrive_expect_tx(bar, (rb ? r.bytes : 0) + (yb ? y.bytes : 0) + (hb ? h.bytes : 0) + (ob ? o.bytes : 0) +
                                       (gb ? g.bytes : 0));
        if (rb) bulk_g2s(to, r.src, r.bytes, bar);
        if (yb) bulk_g2s(to + rb, y.src, y.bytes, bar);
        if (hb) bulk_g2s(to + rb + yb, h.src, h.bytes, bar);
        to += rb + yb + hb;
        if (ob) bulk_g2s(to, o.src, o.bytes, bar);
        if (gb) bulk_g2s(to + ob, g.src, g.bytes, bar);
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

    // Sums over the chunk's rows.  A gate that several rows share: post[] are sum G y^ and
    // sum G over the rows of its group, and at the group's end give its gradient, b (gamma
    // sum G y^ + beta sum G), and their parts of dgamma_post and dbeta_post, b gate times
    // them.  Else post[] are those gradients themselves.
    const bool shared = a.gate && a.gate_rows != 1;
    constexpr int SUMS = FULL ? 2 : 1;
    float2 pre_sum[SUMS][N], post_sum[SUMS][N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        pre_sum[0][k] = post_sum[0][k] = both(0.0f);
        if constexpr (FULL) pre_sum[1][k] = post_sum[1][k] = both(0.0f);
    }
    if (shared) {
        if (a.wants >> kGammaPost & 1) sp.store(part + (int64_t)kGammaPost * a.C, post_sum[0]);
        if (a.wants >> kBetaPost & 1) sp.store(part + (int64_t)kBetaPost * a.C, post_sum[0]);
    }
    auto add = [](float2 *to, const float2 *u, const float2 *w) {
#pragma unroll
        for (int e = 0; e < GP; ++e) to[e] = fma2(u[e], w[e], to[e]);
    };
    auto add1 = [](float2 *to, const float2 *u) {
#pragma unroll
        for (int e = 0; e < GP; ++e) to[e] = add2(u[e], to[e]);
    };

    int64_t q = a.gate_rows ? row0 / a.gate_rows : 0;  // the current group, and the row after it
    int64_t q_end = a.gate_rows ? min((q + 1) * a.gate_rows, a.rows) : a.rows;
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t row = row0; row < row1; ++row) {
        const TR *r_row = static_cast<const TR *>(a.r) + row * a.ld_r,
                 *o_row = static_cast<const TR *>(a.dr_out) + row * a.ld_r;
        const TY *y_row = static_cast<const TY *>(a.y) + row * a.ld_y,
                 *h_row = static_cast<const TY *>(a.dh) + row * a.ld_h,
                 *g_row = static_cast<const TY *>(a.gate) + q * a.C;
        if (RING && (V == 8 || row < a.ring_rows)) {
            if (!mbar_wait(bar0 + 8 * stage, phase, a.status)) {
                drain_ring(bar0, a.stages, stage, phase, min(row1, a.ring_rows) - row, a.status);
                return;
            }
            const uint8_t *from = smem + (size_t)stage * bytes;
            r_row = reinterpret_cast<const TR *>(from + window<V, TR>(a.r, row, a.ld_r, a.C).off);
            from += rb;
            y_row = reinterpret_cast<const TY *>(from + window<V, TY>(a.y, row, a.ld_y, a.C).off);
            from += yb;
            h_row = reinterpret_cast<const TY *>(from + window<V, TY>(a.dh, row, a.ld_h, a.C).off);
            from += hb;
            o_row = reinterpret_cast<const TR *>(from + window<V, TR>(a.dr_out, row, a.ld_r, a.C).off);
            if (gb) g_row = reinterpret_cast<const TY *>(from + ob + window<V, TY>(a.gate, row, a.C, a.C).off);
        }
        constexpr bool KEEP = V * I <= 8 && !FULL;  // y stays in registers
        float2 x[N], g[N], yv[N];  // r', then x^; dh, then G, then t's and dy; y, then y^
        Stats sx{0.0f, 1.0f}, sy{0.0f, 1.0f};
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = yv[k] = both(0.0f);
        if (pre) sp.load(r_row, x);
        if (a.y) sp.load(y_row, yv);
        if (pre || post) stats_of_two<FULL>(sp, x, yv, a, red, sx, sy);
        if (a.dh) sp.load(h_row, g);
        else
#pragma unroll
            for (int k = 0; k < N; ++k) g[k] = both(0.0f);
        if (pre) {
            const float2 rs = both(sx.rstd), mean = both(-sx.mean);
            float2 sg = both(0.0f), sgx = both(0.0f);
#pragma unroll
            for (int i = 0; i < S::G; ++i) {
                float2 *xv = x + i * GP, *gv = g + i * GP, gm[GP], tg = sg, tx = sgx;
                if (a.gamma_pre) sp.load_group(a.gamma_pre, i, gm);
#pragma unroll
                for (int e = 0; e < GP; ++e) xv[e] = mul2(FULL ? add2(xv[e], mean) : xv[e], rs);
                add(pre_sum[0] + i * GP, gv, xv);
                if constexpr (FULL) add1(pre_sum[1] + i * GP, gv);
#pragma unroll
                for (int e = 0; e < GP; ++e) {
                    if (a.gamma_pre) gv[e] = mul2(gv[e], gm[e]);
                    if (FULL) tg = add2(tg, gv[e]);
                    tx = fma2(gv[e], xv[e], tx);
                }
                if (FULL) sg = sp.keep(i, tg, sg);
                sgx = sp.keep(i, tx, sgx);
            }
            gradient<FULL>(sp, g, x, sg, sgx, a.pre == QNN_NORM_LAYER, sx.rstd, a.inv_c, red);
        }
        if (a.dr_out) {
            sp.load(o_row, x);
#pragma unroll
            for (int k = 0; k < N; ++k) g[k] = add2(g[k], x[k]);
        }
        if (a.dr) {
            const float2 f = both(a.a);
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = mul2(f, g[k]);
            sp.store(static_cast<TR *>(a.dr) + row * a.ld_r, x);
        }
        if (a.y) {
            if (!KEEP) sp.load(y_row, yv);
            const float2 rs = both(sy.rstd), mean = both(-sy.mean), f = both(a.b);
            float2 sg = both(0.0f), sgx = both(0.0f);
            TY *gate_out = a.dgate && a.gate_rows == 1 ? static_cast<TY *>(a.dgate) + row * a.C : nullptr;
#pragma unroll
            for (int i = 0; i < S::G; ++i) {
                float2 *xv = yv + i * GP, *gv = g + i * GP, gm[GP], w[GP], tg = sg, tx = sgx;
                if (a.gamma_post) sp.load_group(a.gamma_post, i, gm);
                if (a.gate) sp.load_group(g_row, i, w);
#pragma unroll
                for (int e = 0; e < GP; ++e)
                    if (post) xv[e] = mul2(FULL ? add2(xv[e], mean) : xv[e], rs);
                if (shared) {
                    add(post_sum[0] + i * GP, gv, xv);
                    if constexpr (FULL) add1(post_sum[1] + i * GP, gv);
                }
#pragma unroll
                for (int e = 0; e < GP; ++e) gv[e] = mul2(gv[e], f);
                if (gate_out) {  // b G p
                    float2 t[GP], p[GP];
                    if (FULL && a.beta_post) sp.load_group(a.beta_post, i, p);
#pragma unroll
                    for (int e = 0; e < GP; ++e) {
                        t[e] = a.gamma_post ? mul2(xv[e], gm[e]) : xv[e];
                        if (FULL && a.beta_post) t[e] = add2(t[e], p[e]);
                        t[e] = mul2(t[e], gv[e]);
                    }
                    sp.store_group(gate_out, i, t);
                }
                if (a.gate)
#pragma unroll
                    for (int e = 0; e < GP; ++e) gv[e] = mul2(gv[e], w[e]);
                if (post) {
                    if (!shared) {
                        add(post_sum[0] + i * GP, gv, xv);
                        if constexpr (FULL) add1(post_sum[1] + i * GP, gv);
                    }
#pragma unroll
                    for (int e = 0; e < GP; ++e) {
                        if (a.gamma_post) gv[e] = mul2(gv[e], gm[e]);
                        if (FULL) tg = add2(tg, gv[e]);
                        tx = fma2(gv[e], xv[e], tx);
                    }
                    if (FULL) sg = sp.keep(i, tg, sg);
                    sgx = sp.keep(i, tx, sgx);
                }
            }
            if (post) gradient<FULL>(sp, g, yv, sg, sgx, a.post == QNN_NORM_LAYER, sy.rstd, a.inv_c, red);
        }
        if constexpr (RING) {
            // all threads have read the stage: behind the last reduction, or a barrier for it
            if (!post) __syncthreads();
            if (threadIdx.x == 0 && row + a.stages < row1) ask(row + a.stages, stage);
            if (++stage == a.stages) stage = 0, phase ^= 1;
        }
        if (a.dy) sp.store(static_cast<TY *>(a.dy) + row * a.ld_y, g);
        if (shared && (row + 1 == q_end || row + 1 == row1)) {  // the group ends with this row, or the chunk does
            const bool began = q * a.gate_rows >= row0, whole = began && row + 1 == q_end;
            float *edge = part + (int64_t)(began ? kGateTail : kGateHead) * a.C;
            const TY *gate = static_cast<const TY *>(a.gate) + q * a.C;
            const float2 f = both(a.b);
#pragma unroll
            for (int i = 0; i < S::G; ++i) {
                float2 w[GP], t[GP], o[GP], *s0 = post_sum[0] + i * GP;
                sp.load_group(gate, i, w);
#pragma unroll
                for (int e = 0; e < GP; ++e) w[e] = mul2(w[e], f);
                if (a.wants >> kGammaPost & 1) {
                    float *to = part + (int64_t)kGammaPost * a.C;
                    sp.load_group(to, i, o);
                    add(o, s0, w);
                    sp.store_group(to, i, o);
                }
                if constexpr (FULL)
                    if (a.wants >> kBetaPost & 1) {
                        float *to = part + (int64_t)kBetaPost * a.C;
                        sp.load_group(to, i, o);
                        add(o, post_sum[1] + i * GP, w);
                        sp.store_group(to, i, o);
                    }
                if (a.dgate) {
                    if (a.gamma_post) sp.load_group(a.gamma_post, i, w);
#pragma unroll
                    for (int e = 0; e < GP; ++e) t[e] = a.gamma_post ? mul2(s0[e], w[e]) : s0[e];
                    if constexpr (FULL)
                        if (a.beta_post) {
                            sp.load_group(a.beta_post, i, w);
                            add(t, post_sum[1] + i * GP, w);
                        }
#pragma unroll
                    for (int e = 0; e < GP; ++e) t[e] = mul2(t[e], f);
                    if (whole) sp.store_group(static_cast<TY *>(a.dgate) + q * a.C, i, t);
                    else sp.store_group(edge, i, t);
                }
#pragma unroll
                for (int e = 0; e < GP; ++e) {
                    s0[e] = both(0.0f);
                    if constexpr (FULL) post_sum[1][i * GP + e] = both(0.0f);
                }
            }
        }
        if (row + 1 == q_end) {
            ++q;
            q_end = min(q_end + a.gate_rows, a.rows);
        }
    }
    auto put = [&](int slot, const float2 *v) {
        if (a.wants >> slot & 1) sp.store(part + (int64_t)slot * a.C, v);
    };
    put(kGammaPre, pre_sum[0]);
    if constexpr (FULL) put(kBetaPre, pre_sum[1]);
    if (!shared) {
        put(kGammaPost, post_sum[0]);
        if constexpr (FULL) put(kBetaPost, post_sum[1]);
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
    grid_dependency_wait();  // by blocks without a job too: a grid that waited for nothing could end before the rows'
    if (!param) {
        if (a.by_group) q = job;
        else q = (job + 1) * a.chunk / a.gate_rows;  // the group of the first row behind the boundary
        const int64_t r0 = q * a.gate_rows, r1 = a.gate_rows ? min(r0 + a.gate_rows, a.rows) : a.rows;
        b0 = (int)(r0 / a.chunk);
        b1 = (int)((r1 - 1) / a.chunk) + 1;
        if (b1 - b0 == 1 || (!a.by_group && b0 != job)) return;  // one block's alone, or another boundary's
    }
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

// Whether a LAYER norm or a beta takes part: the kernel with all the sums.
bool back_full(const qnn_block_norm *p)
{
    return p->pre == QNN_NORM_LAYER || p->post == QNN_NORM_LAYER || p->beta_pre || p->beta_post;
}

// Columns of a thread.  16 spread the fixed work of a row (reductions, addresses) over
// more of them, where their sums fit the registers (4096 bf16 columns, RMS: 59 us with
// 16, 70 with 8; LAYER with betas: 116 and 84).  LAYER beyond 4096 columns spills about
// 430 bytes a thread with its 16.
int back_columns(int C, bool full) { return C <= (full ? 4096 : 1024) ? 8 : C <= 8192 ? 16 : 32; }

int back_threads(int C, bool full)
{
    const int per = 32 * back_columns(C, full);
    return (C + per - 1) / per * 32;
}

// Blocks that an SM's registers hold (up to 128 a thread, 64 beyond 8192 columns), 16 at
// most: more blocks are more sums to add.
int back_blocks_per_sm(int C, bool full)
{
    return std::max(1, std::min(16, (C <= 8192 ? 512 : 1024) / back_threads(C, full)));
}

struct BackPlan {
    int64_t chunk;  // rows of a block
    int blocks, stages;
};

BackPlan back_plan(int64_t rows, int C, bool full, int stage)
{
    BackPlan p;
    int per_sm = back_blocks_per_sm(C, full);
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

template <typename TR, typename TY, int V, int I, bool RING, bool FULL>
qnn_status launch_back(BackArgs a, const BackPlan &p, int threads, int stage, cudaStream_t s)
{
    auto kern = block_norm_backward_kernel<TR, TY, V, I, RING, FULL>;
    a.stages = p.stages;
    if (RING) {
        static std::atomic<uint64_t> opted_in{0};
        if (!opt_in_smem(kern, kMaxRing, opted_in, kRingCarveout)) return QNN_ERR_CUDA;
    }
    return launch_dependent(kern, a, p.blocks, threads, RING ? p.stages * stage : 0, s);
}

}  // namespace
}  // namespace qnn

extern "C" size_t qnn_block_norm_backward_workspace_bytes(int64_t rows, int C, const qnn_block_norm *p)
{
    using namespace qnn;
    if (!p || rows < 0 || C <= 0 || C > kMaxC) return 0;
    // the most blocks that any types lead to
    return (size_t)std::min<int64_t>(rows, (int64_t)sm_count() * back_blocks_per_sm(C, back_full(p))) * kSlots * C * sizeof(float);
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
    if (rows == 0 && !sums) return QNN_OK;
    BackArgs a{};
    a.r = r_out, a.y = y, a.gate = p->gate, a.dh = dh, a.dr_out = dr_out, a.dr = dr, a.dy = dy, a.dgate = dgate;
    a.gamma_post = p->gamma_post, a.beta_post = p->beta_post, a.gamma_pre = p->gamma_pre;
    a.ws = static_cast<float *>(workspace);
    // a group reaches no further than the rows, and sums of the two stay in 64 bits (a single
    // row's group keeps the form of shared ones)
    const int64_t gate_rows = std::min(p->gate_rows, std::max<int64_t>(rows, 2));
    a.rows = rows, a.gate_rows = gate_rows, a.C = C, a.post = p->post, a.pre = p->pre;
    a.ld_r = p->ld_r ? p->ld_r : C, a.ld_y = p->ld_y ? p->ld_y : C, a.ld_h = p->ld_h ? p->ld_h : C;
    a.a = p->res_scale, a.b = p->block_scale, a.eps_post = p->eps_post, a.eps_pre = p->eps_pre, a.inv_c = 1.0f / C;
    a.wants = (dgamma_pre ? 1u << kGammaPre : 0) | (dbeta_pre ? 1u << kBetaPre : 0) |
              (dgamma_post ? 1u << kGammaPost : 0) | (dbeta_post ? 1u << kBetaPost : 0);
    a.status = status_word();
    if (!a.status) return QNN_ERR_CUDA;
    const int er = float_bytes(r_dt), ey = float_bytes(y_dt);
    const bool vec = C % 8 == 0 && rows_aligned(a.ld_r, er) && (!y || rows_aligned(a.ld_y, ey)) &&
                     (!dh || rows_aligned(a.ld_h, ey));
    const int rr = vec ? window_room<8>(C, er) : window_room<1>(C, er), yr = vec ? window_room<8>(C, ey) : window_room<1>(C, ey);
    const bool own_gate = p->gate && p->gate_rows == 1, needs_r = dh && p->pre != QNN_NORM_NONE;
    const int stage = (needs_r ? rr : 0) + (y ? yr : 0) + (dh ? yr : 0) + (dr_out ? rr : 0) + (own_gate ? yr : 0);
    const bool ring = C <= kMaxRingC;
    static_assert(5 * ((kMaxRingC * 4 + 30) & ~15) <= kMaxRing, "a stage of five fp32 windows has to fit");
    a.ring_rows = rows;
    if (!vec) {
        a.ring_rows = ring_rows(rows, a.ld_r, er);
        if (y) a.ring_rows = std::min(a.ring_rows, ring_rows(rows, a.ld_y, ey));
        if (dh) a.ring_rows = std::min(a.ring_rows, ring_rows(rows, a.ld_h, ey));
        if (own_gate) a.ring_rows = std::min(a.ring_rows, ring_rows(rows, C, ey));
    }
    const bool full = back_full(p), eight = back_columns(C, full) == 8;
    const int threads = back_threads(C, full);
    const BackPlan plan = back_plan(rows, C, full, ring ? stage : 0);
    a.chunk = plan.chunk;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows > 0) {
        qnn_status done = QNN_OK;
        with_types(r_dt, y_dt, [&](auto tr, auto ty) {
            using TR = decltype(tr);
            using TY = decltype(ty);
            if (ring && vec && eight)
                done = full ? launch_back<TR, TY, 8, 1, true, true>(a, plan, threads, stage, s)
                            : launch_back<TR, TY, 8, 1, true, false>(a, plan, threads, stage, s);
            else if (ring && vec)
                done = full ? launch_back<TR, TY, 8, 2, true, true>(a, plan, threads, stage, s)
                            : launch_back<TR, TY, 8, 2, true, false>(a, plan, threads, stage, s);
            else if (ring && eight) done = launch_back<TR, TY, 1, 8, true, true>(a, plan, threads, stage, s);
            else if (ring)
                done = full ? launch_back<TR, TY, 1, 16, true, true>(a, plan, threads, stage, s)
                            : launch_back<TR, TY, 1, 16, true, false>(a, plan, threads, stage, s);
            else if (vec) done = launch_back<TR, TY, 8, 4, false, true>(a, plan, threads, 0, s);
            else done = launch_back<TR, TY, 1, 32, false, true>(a, plan, threads, 0, s);
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
    f.dgate = dgate, f.gate_dt = y_dt, f.rows = rows, f.gate_rows = gate_rows, f.chunk = a.chunk, f.C = C;
    f.blocks = plan.blocks;
    int64_t jobs = 0;
    if (dgate && f.blocks > 1) {
        const int64_t groups = gate_rows ? (rows + gate_rows - 1) / gate_rows : 1;
        f.by_group = groups < f.blocks;
        jobs = gate_rows == 1 ? 0 : f.by_group ? groups : f.blocks - 1;
    }
    const dim3 grid((C + 31) / 32, (unsigned)(f.sums + jobs));
    if (grid.y == 0) return QNN_OK;
    return launch_dependent(block_norm_finish_kernel, f, grid, kFinishWarps * 32, 0, s);
}
