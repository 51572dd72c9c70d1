// qnn_kv_attn.cu -- q_kv_attn: attention of the newest tokens over the quantised cache.
#include "qnn_kv.cuh"

namespace qnn {
namespace {

struct KvAttnArgs {
    KvArgs c;
    const void *q;
    void *out;
    float *lse;
    const uint32_t *mask;
    int64_t ld_q, ld_out;
    float scale_log2;  // scale * log2(e)
    int heads_q, group, mask_words;
};

constexpr int kThreads = 128;

// One block for a row and head, a token to a warp at a time.
template <typename T, bool U4>
__global__ void __launch_bounds__(kThreads) kv_attn_kernel(const __grid_constant__ KvAttnArgs a)
{
    const KvArgs &c = a.c;
    __shared__ float part[4][256 + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = c.D / 32;
    const int64_t row = blockIdx.x;
    const int hq = blockIdx.y, h = hq / a.group;
    grid_dependency_launch();
    grid_dependency_wait();
    int b = 0;
    if (c.starts) while (b < c.batch && c.starts[b + 1] <= row) ++b;
    else b = (int)(row / c.tokens);
    if (b >= c.batch) return;
    const KvSeq s = kv_seq(c, b);
    const int64_t t = row - s.first;
    if (s.T < 0 || t < 0 || t >= s.T) return;
    float q[8], acc[8], m = -INFINITY, l = 0.0f;
    for (int e = 0; e < n; ++e) {
        q[e] = to_f32(static_cast<const T *>(a.q)[row * a.ld_q + (int64_t)hq * c.D + lane * n + e]);
        acc[e] = 0.0f;
    }
    for (int pos = warp; pos < s.len; pos += 4) {
        const int j = pos - (s.len - s.T);
        if (j >= 0) {
            if (!a.mask) {
                if (j > t) continue;
            } else if (j >= 32 * a.mask_words || !(a.mask[row * a.mask_words + j / 32] >> (j % 32) & 1u)) {
                continue;
            }
        }
        const int pg = kv_page(c, b, pos / c.page), slot = pos % c.page;
        if (pg < 0) continue;
        const uint8_t *head = c.pages + pg * c.page_bytes + (int64_t)h * c.head_bytes;
        const uint32_t *words = reinterpret_cast<const uint32_t *>(head + 2 * c.page * c.row_bytes);
        const uint32_t wk = words[slot], wv = words[c.page + slot];
        auto code = [&](const uint8_t *r, int d) {
            if constexpr (U4) return (float)(r[16 * kv_chunk(c.chunks, slot, d / 32) + d % 32 / 2] >> (4 * (d & 1)) & 15);
            else return (float)r[16 * kv_chunk(c.chunks, slot, d / 16) + d % 16];
        };
        const float zk = U4 ? (float)(wk & 15u) : 128.0f, zv = U4 ? (float)(wv & 15u) : 128.0f;
        const float sk = __uint_as_float(U4 ? wk & 0xffff0000u : wk), sv = __uint_as_float(U4 ? wv & 0xffff0000u : wv);
        float x = 0.0f;
        for (int e = 0; e < n; ++e) x = __fmaf_rn(q[e], code(head + slot * c.row_bytes, lane * n + e) - zk, x);
        for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= sk * a.scale_log2;
        const float up = fmaxf(m, x), f = m == -INFINITY ? 0.0f : exp2f(m - up), p = exp2f(x - up);
        m = up;
        l = l * f + p;
        for (int e = 0; e < n; ++e)
            acc[e] = acc[e] * f + p * (code(head + (c.page + slot) * c.row_bytes, lane * n + e) - zv) * sv;
    }
    for (int e = 0; e < n; ++e) part[warp][lane * n + e] = acc[e];
    if (lane == 0) part[warp][256] = m, part[warp][257] = l;
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, part[w][256]);
    for (int w = 0; w < 4; ++w) sum += part[w][257] * (part[w][256] == top ? 1.0f : exp2f(part[w][256] - top));
    for (int d = threadIdx.x; d < c.D; d += kThreads) {
        float o = 0.0f;
        for (int w = 0; w < 4; ++w) o += part[w][d] * (part[w][256] == top ? 1.0f : exp2f(part[w][256] - top));
        static_cast<T *>(a.out)[row * a.ld_out + (int64_t)hq * c.D + d] = from_f32<T>(sum == 0.0f ? 0.0f : o / sum);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[row * a.heads_q + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
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
    return 16;
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
    const dim3 grid((unsigned)a.c.rows, (unsigned)heads_q);
    const bool u4 = g->kv_dt == QNN_U4;
    if (x_dt == QNN_F16)
        return u4 ? kv_launch(kv_attn_kernel<__half, true>, grid, kThreads, 0, (cudaStream_t)stream, a)
                  : kv_launch(kv_attn_kernel<__half, false>, grid, kThreads, 0, (cudaStream_t)stream, a);
    return u4 ? kv_launch(kv_attn_kernel<__nv_bfloat16, true>, grid, kThreads, 0, (cudaStream_t)stream, a)
              : kv_launch(kv_attn_kernel<__nv_bfloat16, false>, grid, kThreads, 0, (cudaStream_t)stream, a);
}
