// qnn_kv_attn.cu -- q_kv_attn: attention of the newest tokens over the quantised cache.  The
// entry, the choice of the kernel, and the kernel that joins the parts of items that several
// blocks had.
#include "qnn_kv_attn.cuh"

namespace qnn {
namespace {

constexpr int kJoinThreads = 128, kJoinRows = 8;

// A block joins kJoinRows rows of the item that begins in block blockIdx.x's share and ends in a
// later one's, if there is one.
__global__ void __launch_bounds__(kJoinThreads) kv_attn_join_kernel(const __grid_constant__ KvAttnArgs a, int rows,
                                                                    int channels, float weight_unit)
{
    __shared__ float factor[kJoinRows][kAttnMaxBlocks], tops[kJoinRows], totals[kJoinRows], unit_of[kJoinRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = blockIdx.x, r0 = blockIdx.y * kJoinRows;
    grid_dependency_launch();
    grid_dependency_wait();
    const volatile int *record = reinterpret_cast<const int *>(a.ws) + block * kAttnRecord;
    if (!record[0]) return;
    const int b = record[1], rt = record[2], head = record[3], n = record[4] - block + 1;
    const KvSeq s = kv_seq(a.c, b);
    const int width = (int)min((int64_t)rows, (int64_t)s.T * a.group - (int64_t)rt * rows);
    if (r0 >= width) return;
    auto slot = [&](int k) { return attn_slot(a, block + k, k == 0 ? 1 : 0, rows, channels); };
    for (int r = warp; r < kJoinRows && r0 + r < width; r += kJoinThreads / 32) {
        const int64_t stat = (int64_t)rows * channels + 2 * (r0 + r);
        float top = -INFINITY, unit = 0.0f, total = 0.0f;
        for (int k = lane; k < n; k += 32) {
            top = fmaxf(top, slot(k)[stat]);
            unit = fmaxf(unit, slot(k)[(int64_t)rows * (channels + 2)]);
        }
        for (int d = 16; d > 0; d /= 2) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            unit = fmaxf(unit, __shfl_xor_sync(0xffffffffu, unit, d));
        }
        for (int k = lane; k < n; k += 32) {
            const float m = slot(k)[stat], f = m == top ? 1.0f : ex2(m - top);
            total = __fmaf_rn(slot(k)[stat + 1], f, total);
            // units are powers of two: the quotient by a reciprocal is exact
            factor[r][k] = f * (slot(k)[(int64_t)rows * (channels + 2)] * __uint_as_float(0x7f000000u - __float_as_uint(unit)));
        }
        for (int d = 16; d > 0; d /= 2) total += __shfl_xor_sync(0xffffffffu, total, d);
        if (lane == 0) tops[r] = top, totals[r] = total, unit_of[r] = unit;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kJoinRows * a.c.D / 2; i += kJoinThreads) {
        const int r = i / (a.c.D / 2), d = 2 * (i - r * (a.c.D / 2));
        if (r0 + r >= width) break;
        float v0 = 0.0f, v1 = 0.0f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float2 v = *reinterpret_cast<const float2 *>(slot(k) + (int64_t)(r0 + r) * channels + d);
            v0 = __fmaf_rn(v.x, factor[r][k], v0), v1 = __fmaf_rn(v.y, factor[r][k], v1);
        }
        attn_store(a, s.first, head, rt * rows + r0 + r, d, v0, v1, tops[r], totals[r], unit_of[r] * weight_unit);
    }
}

bool many_rows(const KvArgs &c, int group) { return c.D <= 128 && (int64_t)c.tokens * group > 32; }

AttnPlan attn_plan(const KvArgs &c, int group)
{
    return many_rows(c, group) ? attn_rows_plan(c, group) : attn_few_plan(c, group);
}

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
    const qnn::AttnPlan p = qnn::attn_plan(c, heads_q / g->heads);
    return 4 * (size_t)(p.blocks * (qnn::kAttnRecord + 2 * qnn::attn_slot_floats(p.rows, p.channels)));
}

extern "C" qnn_status q_kv_attn(const void *q, qnn_dtype x_dt, int64_t ld_q, int heads_q, const qnn_kv_geom *g,
                                const qnn_kv_seqs *seqs, float scale, const uint32_t *mask, int mask_words, void *out,
                                int64_t ld_out, float *lse, void *workspace, size_t workspace_bytes, qnn_stream_t stream)
{
    using namespace qnn;
    KvAttnArgs a = {};
    const qnn_status st = kv_args(g, seqs, &a.c);
    if (st != QNN_OK) return st;
    if (!heads_ok(g, heads_q) || !(scale - scale == 0.0f) || mask_words < 0 || (mask && mask_words == 0))
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
    a.scale_log2 = (float)(scale * 1.4426950408889634);
    a.heads_q = heads_q;
    a.group = heads_q / g->heads;
    if (!(a.c.status = status_word())) return QNN_ERR_CUDA;
    const AttnPlan p = attn_plan(a.c, a.group);
    a.blocks = p.blocks;
    a.bf16 = x_dt == QNN_BF16;
    a.ws = static_cast<float *>(workspace);
    a.per16 = g->page / 16;
    a.magic16 = (int)(((1ull << 32) + a.per16 - 1) / a.per16);
    const qnn_status sent = (many_rows(a.c, a.group) ? launch_attn_rows : launch_attn_few)(a, p, g->kv_dt == QNN_U4,
                                                                                          (cudaStream_t)stream);
    if (sent != QNN_OK) return sent;
    return kv_launch(kv_attn_join_kernel, dim3((unsigned)p.blocks, (unsigned)(p.rows / kJoinRows)), kJoinThreads, 0,
                     (cudaStream_t)stream, a, p.rows, p.channels, kAttnWeightUnit);
}
