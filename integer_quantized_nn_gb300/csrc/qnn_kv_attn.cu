// qnn_kv_attn.cu -- q_kv_attn: attention of the newest tokens over the quantised cache.  The
// entry, the choice of the kernel, and the kernel that joins the parts of items that several
// blocks had.
#include "qnn_kv_attn.cuh"

namespace qnn {
namespace {

// What joins parts of the online softmax: the maximum, the power of two that the values are in, sums.
template <int V>
struct Joined {
    float top = -INFINITY, unit = 0.0f, total = 0.0f, sum[V] = {};

    // what there is, in a larger maximum and unit
    __device__ __forceinline__ void move(float new_top, float new_unit)
    {
        const float f = top == new_top ? 1.0f : ex2(top - new_top), g = f * (unit * pow2_inverse(new_unit));
        total *= f;
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] *= g;
        top = new_top, unit = new_unit;
    }
};

template <int V>
__device__ __forceinline__ void load_channels(const float *p, float (&x)[V])
{
    if constexpr (V == 2) {
        const float2 w = *reinterpret_cast<const float2 *>(p);
        x[0] = w.x, x[1] = w.y;
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 w = *reinterpret_cast<const float4 *>(p + e);
            x[e] = w.x, x[e + 1] = w.y, x[e + 2] = w.z, x[e + 3] = w.w;
        }
    }
}

constexpr int kJoinWarps = 8;

// Block (x, y) joins up to 8 rows of the item that begins in block x's share and ends in a later
// one's, if there is one.  Where fewer rows are left than warps, several warps have a row: each joins
// every so manieth part, the first of them what all have (38 parts a row, cold: 9.5 us, 21 with one
// warp).  Lane k has the statistics of a warp's part k (and k + 32, ..), all lanes the channels.  A chain of
// reads that wait for one another is all that takes time here, so only the record is waited for
// before the first parts are asked for.
template <int V>  // channels of a lane: 2, 4 or 8
__global__ void __launch_bounds__(kJoinWarps * 32) kv_attn_join_kernel(const __grid_constant__ KvAttnArgs a, int rows)
{
    constexpr int channels = 32 * V, kWarps = kJoinWarps, kAtOnce = 4;
    __shared__ float values[kWarps][channels];
    __shared__ float stats[kWarps][3];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = blockIdx.x;
    grid_dependency_launch();
    grid_dependency_wait();
    int4 rec;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(rec.x), "=r"(rec.y), "=r"(rec.z), "=r"(rec.w)
                 : "l"(reinterpret_cast<const int4 *>(a.ws) + 2 * block));
    const int left = rec.w - (int)blockIdx.y * kWarps;
    if (rec.x < 0 || left <= 0) return;
    const int64_t first = *reinterpret_cast<const volatile int64_t *>(reinterpret_cast<const int4 *>(a.ws) + 2 * block + 1);
    // a power of two of warps to a row
    const int shift = left >= kWarps ? 0 : __clz(left > 1 ? left - 1 : 0) - __clz(kWarps - 1);
    const int each = 1 << shift, sub = warp & (each - 1), row = blockIdx.y * kWarps + (warp >> shift);
    const bool live = row < rec.w;
    const int n = live ? (rec.x - block + 1 - sub + each - 1) >> shift : 0;  // parts of this warp
    const float *part0 = attn_slot(a, block, 1, rows, channels), *part1 = attn_slot(a, block + 1, 0, rows, channels);
    const int64_t pitch = 2 * attn_slot_floats(rows, channels);  // between the parts after the first
    auto part = [&](int i) {
        const int k = (i << shift) + sub;
        return k == 0 ? part0 : part1 + (k - 1) * pitch;
    };
    const int d = lane * V;
    Joined<V> j;
    for (int i0 = 0; i0 < n; i0 += 32) {  // 32 parts at a time
        const int here = min(32, n - i0);
        float x[kAtOnce][V], m = -INFINITY, l = 0.0f, u = 0.0f;
        auto ask = [&](int i) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (i + k < here) load_channels(part(i0 + i + k) + (int64_t)row * channels + d, x[k]);
        };
        if (lane < here) {
            const float *p = part(i0 + lane) + (int64_t)rows * channels;
            const float2 ml = *reinterpret_cast<const float2 *>(p + 2 * row);
            m = ml.x, l = ml.y, u = p[2 * rows + row];
        }
        ask(0);
        float top = fmaxf(j.top, m), unit = fmaxf(j.unit, u);
#pragma unroll
        for (int b = 16; b > 0; b /= 2) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
            unit = fmaxf(unit, __shfl_xor_sync(0xffffffffu, unit, b));
        }
        j.move(top, unit);
        const float f = m == top ? 1.0f : ex2(m - top), g = lane < here ? f * (u * pow2_inverse(unit)) : 0.0f;
        float t = lane < here ? l * f : 0.0f;
#pragma unroll
        for (int b = 16; b > 0; b /= 2) t += __shfl_xor_sync(0xffffffffu, t, b);
        j.total += t;
        for (int i = 0; i < here; i += kAtOnce) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float w = __shfl_sync(0xffffffffu, g, i + k);
                if (i + k >= here) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) j.sum[e] = __fmaf_rn(x[k][e], w, j.sum[e]);
            }
            ask(i + kAtOnce);
        }
    }
    if (each > 1) {
        if (sub) {
#pragma unroll
            for (int e = 0; e < V; ++e) values[warp][e * 32 + lane] = j.sum[e];
            if (lane == 0) stats[warp][0] = j.top, stats[warp][1] = j.unit, stats[warp][2] = j.total;
        }
        __syncthreads();
        if (sub) return;
        for (int w = warp + 1; w < warp + min(each, rec.x - block + 1); ++w) {
            Joined<V> o;
            o.top = stats[w][0], o.unit = stats[w][1], o.total = stats[w][2];
#pragma unroll
            for (int e = 0; e < V; ++e) o.sum[e] = values[w][e * 32 + lane];
            const float top = fmaxf(j.top, o.top), unit = fmaxf(j.unit, o.unit);
            j.move(top, unit), o.move(top, unit);
            j.total += o.total;
#pragma unroll
            for (int e = 0; e < V; ++e) j.sum[e] += o.sum[e];
        }
    }
    if (!live) return;
    const float total = j.total, unit = j.unit, top = j.top;
    const float (&sum)[V] = j.sum;
    const float by = total == 0.0f ? 0.0f : kAttnWeightUnit * unit / total;
    const int r = rec.z + row, tok = r / a.group, hq = rec.y * a.group + (r - tok * a.group);
    if (d < a.c.D) {
        uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + (first + tok) * a.ld_out +
                                                     (int64_t)hq * a.c.D + d);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) out[e] = attn_pack(a, sum[2 * e] * by, sum[2 * e + 1] * by);
    }
    if (a.lse && lane == 0) a.lse[(first + tok) * a.heads_q + hq] = attn_lse(top, total);
}

// Where the tensor memory's kernel takes over.  Few against many rows, in 8 bits, 32 heads of q on 8 (D = 256: 64), us:
//   16 sequences of 4096, D = 128:  8 rows 43 / 58, and 16 and 32 rows of the second 58 and 59
//   1 of 512, D = 128:              8 rows 10.9 / 13.1
//   16 of 4096, D = 64:             8 rows 30 / 47, 16 rows 40 / 47, 32 rows 58 / 49; 32 heads on 32 over 1024, 16 rows
//                                   49 / 67
//   16 of 4096, D = 256:            8 rows 65 / 107, 16 rows 71 / 109, 32 rows 122 / 112, 64 rows 222 / 118; 1 of 512,
//                                   32 rows 16.0 / 17.4
// For D > 128 the two cross below 32 rows where sequences are long, and above where they are short.
int most_few_rows(const KvArgs &c) { return c.D <= 64 ? 16 : c.D <= 128 ? 8 : 32; }

bool many_rows(const KvArgs &c, int group)
{
    // with D > 128 the sums of a longer batch have no room
    return (int64_t)c.tokens * group > most_few_rows(c) && (c.D <= 128 || c.batch <= 2048);
}

// A batch in which most sequences have far fewer newest tokens than the longest (prompts beside sequences that
// decode) goes through both kernels, each with the sequences that suit it.  The host knows the tokens' number and
// the most of one; where the mean is below a quarter of the most, two more launches (about 4 us) are worth it: 63
// sequences of 4096 with one token beside one with 512, 32 heads on 8, D = 128, 8 bits: 195 us, 344 by one kernel.
struct AttnPlans {
    AttnPlan plan[2];
    int t_min[2], t_max[2], count;
    bool many[2];
};

AttnPlans attn_plans(const KvArgs &c, int group)
{
    AttnPlans p;
    const int few = most_few_rows(c) / group;  // tokens of a sequence with few rows
    p.count = 1;
    p.many[0] = many_rows(c, group);
    p.plan[0] = p.many[0] ? attn_rows_plan(c, group) : attn_few_plan(c, group);
    p.t_min[0] = 0, p.t_max[0] = c.tokens;
    if (p.many[0] && c.starts && few > 0 && 4 * c.rows <= (int64_t)c.batch * c.tokens) {
        KvArgs rest = c;
        rest.tokens = few;
        p.count = 2;
        p.many[1] = false;
        p.plan[1] = attn_few_plan(rest, group);
        p.t_min[0] = few + 1;
        p.t_min[1] = 0, p.t_max[1] = few;
    }
    return p;
}

int64_t workspace_floats(const AttnPlan &p) { return p.blocks * (kAttnRecord + 2 * attn_slot_floats(p.rows, p.channels)); }

bool heads_ok(const qnn_kv_geom *g, int heads_q)
{
    return heads_q > 0 && heads_q % g->heads == 0 && heads_q / g->heads <= 1024;
}

}  // namespace
}  // namespace qnn

extern "C" size_t qnn_kv_attn_workspace_bytes(const qnn_kv_geom *g, const qnn_kv_seqs *seqs, int heads_q)
{
    qnn::KvArgs c;
    if (qnn::kv_args(g, seqs, &c) != QNN_OK || !qnn::heads_ok(g, heads_q)) return 0;
    const qnn::AttnPlans p = qnn::attn_plans(c, heads_q / g->heads);
    size_t n = 0;
    for (int i = 0; i < p.count; ++i) n += 4 * (size_t)qnn::workspace_floats(p.plan[i]);
    return n;
}

extern "C" qnn_status q_kv_attn(const void *q, qnn_dtype x_dt, int64_t ld_q, int heads_q, const qnn_kv_geom *g,
                                const qnn_kv_seqs *seqs, float scale, const uint32_t *mask, int mask_words, void *out,
                                int64_t ld_out, float *lse, void *workspace, size_t workspace_bytes, qnn_stream_t stream)
{
    using namespace qnn;
    KvAttnArgs a = {};
    const qnn_status st = kv_args(g, seqs, &a.c);
    if (st != QNN_OK) return st;
    const float scale_log2 = (float)(scale * 1.4426950408889634);
    if (!heads_ok(g, heads_q) || !(scale_log2 - scale_log2 == 0.0f) || mask_words < 0 || (mask && mask_words == 0))
        return QNN_ERR_INVALID_ARG;
    if (x_dt != QNN_F16 && x_dt != QNN_BF16) return QNN_ERR_UNSUPPORTED;
    const int64_t width = (int64_t)heads_q * g->D, most = INT64_MAX / 8 / std::max<int64_t>(1, a.c.rows);
    a.ld_q = ld_q ? ld_q : width;
    a.ld_out = ld_out ? ld_out : width;
    if (a.ld_q < width || a.ld_out < width || a.ld_q > most || a.ld_out > most) return QNN_ERR_INVALID_ARG;
    if ((int64_t)a.c.tokens * (heads_q / g->heads) > INT32_MAX - 256) return QNN_ERR_UNSUPPORTED;
    if (a.c.batch == 0 || a.c.rows == 0) return QNN_OK;
    if (!q || !out || !workspace || workspace_bytes < qnn_kv_attn_workspace_bytes(g, seqs, heads_q))
        return QNN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || a.ld_q % 8 || a.ld_out % 8 ||
        (reinterpret_cast<uintptr_t>(mask) & 3u) || (reinterpret_cast<uintptr_t>(lse) & 3u))
        return QNN_ERR_ALIGNMENT;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.mask = mask;
    a.mask_words = mask_words;
    a.scale_log2 = scale_log2;
    a.heads_q = heads_q;
    a.group = heads_q / g->heads;
    if (!(a.c.status = status_word())) return QNN_ERR_CUDA;
    a.bf16 = x_dt == QNN_BF16;
    a.ws = static_cast<float *>(workspace);
    const AttnPlans plans = attn_plans(a.c, a.group);
    for (int i = 0; i < plans.count; ++i) {
        const AttnPlan &p = plans.plan[i];
        a.blocks = p.blocks;
        a.t_min = plans.t_min[i], a.t_max = plans.t_max[i];
        qnn_status sent = (plans.many[i] ? launch_attn_rows : launch_attn_few)(a, p, g->kv_dt == QNN_U4, (cudaStream_t)stream);
        if (sent != QNN_OK) return sent;
        const dim3 grid((unsigned)p.blocks, (unsigned)(p.rows / kJoinWarps));
        auto join = p.channels == 64    ? kv_attn_join_kernel<2>
                    : p.channels == 128 ? kv_attn_join_kernel<4>
                                        : kv_attn_join_kernel<8>;
        sent = kv_launch(join, grid, kJoinWarps * 32, 0, (cudaStream_t)stream, a, p.rows);
        if (sent != QNN_OK) return sent;
        a.ws += workspace_floats(p);
    }
    return QNN_OK;
}
