// qnn_kv.cu -- the cache of keys and values: quantised as it is written (q_kv_write), read
// back (q_kv_read), and its accepted tokens kept (q_kv_keep).
//
// All three move bytes.  A group of lanes, one for each 8 channels, has a token's head of K or
// V at a time: maxima by shuffles inside the group, one IEEE division for the scale and one for
// each value (so that codes are those of the definition, ties included).  A warp asks for all
// its values before it looks up where they go.
#include "qnn_kv.cuh"

namespace qnn {

qnn_status kv_args(const qnn_kv_geom *g, const qnn_kv_seqs *q, KvArgs *a)
{
    if (!kv_geom_ok(g) || !q) return QNN_ERR_INVALID_ARG;
    if (q->batch < 0 || q->rows < 0 || q->tokens < 0 || q->num_pages < 0 || q->ld_table < 0 ||
        q->num_pages > INT32_MAX || q->rows > INT32_MAX || q->ld_table > INT32_MAX)
        return QNN_ERR_INVALID_ARG;
    if (!q->starts && q->rows != (int64_t)q->batch * q->tokens) return QNN_ERR_INVALID_ARG;
    if (q->batch > kKvMaxBatch) return QNN_ERR_UNSUPPORTED;
    if (q->batch > 0 && (!q->lens || (q->ld_table > 0 && !q->table) || (q->num_pages > 0 && !q->pages)))
        return QNN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q->pages) & 127u) || (reinterpret_cast<uintptr_t>(q->table) & 3u) ||
        (reinterpret_cast<uintptr_t>(q->lens) & 3u) || (reinterpret_cast<uintptr_t>(q->starts) & 3u))
        return QNN_ERR_ALIGNMENT;
    a->pages = static_cast<uint8_t *>(q->pages);
    a->table = q->table;
    a->lens = q->lens;
    a->starts = q->starts;
    a->ld_table = q->ld_table;
    a->rows = q->rows;
    a->num_pages = (int)q->num_pages;
    a->batch = q->batch;
    a->tokens = q->tokens;
    a->heads = g->heads;
    a->D = g->D;
    a->page = g->page;
    a->row_bytes = kv_row_bytes(*g);
    a->chunks = a->row_bytes / 16;
    a->head_bytes = g->page * (2 * a->row_bytes + 8);
    a->page_bytes = (int64_t)a->head_bytes * g->heads;
    a->status = nullptr;
    return QNN_OK;
}

namespace {

constexpr int kWarps = 8, kUnroll = 4;  // items of a group at a time

struct KvIoArgs {
    KvArgs c;
    const void *k, *v;
    int64_t ld_k, ld_v;
    int parts;  // of a row: each 2 * heads / parts items, kUnroll to a group
    int vec;    // rows of k and v start on 16-byte boundaries
};

// The place of a row: its position's page and offset in it; page -1: none.
struct Place {
    int page, slot;  // slot: the token in the page
    int seq;         // 0: no sequence has the row
};

// The sequence whose rows hold `row`: the number of starts[1 .. batch] that are <= row, by a warp.
// (Where they descend the answer is some sequence, and what follows is checked.)
__device__ __forceinline__ int seq_of_row(const KvArgs &a, int64_t row, int lane)
{
    if (!a.starts) return (int)(row / a.tokens);
    int lo = 0, n = a.batch;  // the answer is in lo .. lo + n
    const volatile int32_t *st = a.starts + 1;
    while (n > 0) {
        const int step = (n + 31) / 32, at = (lane + 1) * step - 1;
        const int below = __popc(__ballot_sync(0xffffffffu, at < n && st[lo + at] <= row)) * step;
        lo += below;
        n = min(n - below, step - 1);
    }
    return lo;
}

__device__ __forceinline__ Place place_of(const KvArgs &a, int64_t row, int lane)
{
    Place p = {-1, 0, 0};
    const int b = seq_of_row(a, row, lane);
    if (b >= a.batch) return p;
    const KvSeq s = kv_seq(a, b);
    const int64_t t = row - s.first;
    if (s.T < 0 || t < 0 || t >= s.T) return p;
    p.seq = 1;
    const int64_t pos = s.len - s.T + t;
    if (pos < 0) return p;
    p.page = kv_page(a, b, (int)(pos / a.page));
    p.slot = (int)(pos % a.page);
    return p;
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, int vec, float (&x)[8])
{
    if (vec) {
        uint4 w[sizeof(T) / 2];
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                         : "l"(reinterpret_cast<const uint4 *>(p) + i));
        }
        const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32(p[i]);
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, int vec, const float (&x)[8])
{
    if (vec) {
        uint4 w[sizeof(T) / 2];
        T *e = reinterpret_cast<T *>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(x[i]);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(x[i]);
    }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.4028235e38f; }  // false for NaN

// W lanes have an item's channels, 8 each; `live`: this lane has some.
template <int W>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int d = W / 2; d > 0; d /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

template <typename T, bool U4, int W>
__global__ void __launch_bounds__(kWarps * 32) kv_write_kernel(const __grid_constant__ KvIoArgs a)
{
    const KvArgs &c = a.c;
    constexpr int G = 32 / W;  // items of a warp at a time
    const int lane = threadIdx.x & 31, group = lane / W, j = lane % W, d0 = 8 * j;
    const bool live = d0 < c.D;
    grid_dependency_launch();
    grid_dependency_wait();
    const int64_t units = c.rows * a.parts;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
        const int64_t row = u / a.parts;
        const int first = (int)(u - row * a.parts) * kUnroll * G + group;
        float x[kUnroll][8];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int item = first + i * G;  // K's heads, then V's
            if (item < 2 * c.heads && live) {
                const bool is_v = item >= c.heads;
                const int64_t at = row * (is_v ? a.ld_v : a.ld_k) + (item - (is_v ? c.heads : 0)) * c.D + d0;
                load8(static_cast<const T *>(is_v ? a.v : a.k) + at, a.vec, x[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
            }
        }
        const Place p = place_of(c, row, lane);
        if (p.page < 0) continue;
        uint8_t *base = c.pages + p.page * c.page_bytes;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int item = first + i * G;
            float hi = 0.0f, lo = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!finite(x[i][e])) continue;
                hi = fmaxf(hi, U4 ? x[i][e] : fabsf(x[i][e]));
                if (U4) lo = fmaxf(lo, -x[i][e]);
            }
            hi = group_max<W>(hi);
            if (U4) lo = group_max<W>(lo);  // -min
            float s, z = 0.0f;
            if constexpr (U4) {
                s = __bfloat162float(__float2bfloat16_rn(__fadd_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f))));
                if (s > 0.0f) z = fminf(rintf(__fdiv_rn(lo, s)), 15.0f);
            } else {
                s = __fdiv_rn(hi, 127.0f);
            }
            // By a product with 1 / s first: that is within 2^-21 of the quotient, relatively, and so the same
            // integer but near a tie (and where s or a value is out of the ordinary): then by division.
            uint32_t q[8];
            const float per = __fdiv_rn(1.0f, s);
            bool plain = s > 1e-30f;
            const float zero = 12582912.0f + (U4 ? z : 128.0f);  // 1.5 * 2^23 + the code of zero: integers in its low bits
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = __fmul_rn(x[i][e], per), r = __fadd_rn(t, 12582912.0f);
                plain = plain && fabsf(__fadd_rn(t, -__fadd_rn(r, -12582912.0f))) < 0.4999f;
                q[e] = __float_as_uint(__fadd_rn(r, zero - 12582912.0f)) & 0xffu;
                if constexpr (U4) q[e] = min(max((int)(int8_t)q[e], 0), 15);
            }
            if (!plain) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float r = s > 0.0f && x[i][e] == x[i][e] ? rintf(__fdiv_rn(x[i][e], s)) : 0.0f;
                    if constexpr (U4) q[e] = (uint32_t)fminf(fmaxf(__fadd_rn(r, z), 0.0f), 15.0f);
                    else q[e] = (uint32_t)(fminf(fmaxf(r, -127.0f), 127.0f) + 128.0f);
                }
            }
            if (item >= 2 * c.heads || !live) continue;
            const bool is_v = item >= c.heads;
            uint8_t *head = base + (int64_t)(item - (is_v ? c.heads : 0)) * c.head_bytes;
            uint8_t *to = head + (is_v ? c.page * c.row_bytes : 0) + p.slot * c.row_bytes;
            if constexpr (U4) {
                uint32_t w = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) w |= q[e] << (4 * e);
                *reinterpret_cast<uint32_t *>(to + 16 * kv_chunk(c.chunks, p.slot, j / 4) + 4 * (j % 4)) = w;
            } else {
                const uint32_t w0 = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
                const uint32_t w1 = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
                *reinterpret_cast<uint2 *>(to + 16 * kv_chunk(c.chunks, p.slot, j / 2) + 8 * (j % 2)) =
                    make_uint2(w0, w1);
            }
            if (j == 0) {
                const uint32_t word = U4 ? __float_as_uint(s) | (uint32_t)z : __float_as_uint(s);
                reinterpret_cast<uint32_t *>(head + 2 * c.page * c.row_bytes)[(is_v ? c.page : 0) + p.slot] = word;
            }
        }
    }
}

template <typename T, bool U4, int W>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const __grid_constant__ KvIoArgs a)
{
    const KvArgs &c = a.c;
    constexpr int G = 32 / W;
    const int lane = threadIdx.x & 31, group = lane / W, j = lane % W, d0 = 8 * j;
    const bool live = d0 < c.D;
    grid_dependency_launch();
    grid_dependency_wait();
    const int64_t units = c.rows * a.parts;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
        const int64_t row = u / a.parts;
        const int first = (int)(u - row * a.parts) * kUnroll * G + group;
        const Place p = place_of(c, row, lane);
        if (!p.seq || !live) continue;
        uint32_t w[kUnroll][2], word[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int item = first + i * G;
            const bool is_v = item >= c.heads;
            w[i][0] = w[i][1] = U4 ? 0 : 0x80808080u;
            word[i] = 0;
            if (item >= 2 * c.heads || p.page < 0) continue;
            const uint8_t *head = c.pages + p.page * c.page_bytes + (int64_t)(item - (is_v ? c.heads : 0)) * c.head_bytes;
            const uint8_t *from = head + (is_v ? c.page * c.row_bytes : 0) + p.slot * c.row_bytes;
            if constexpr (U4) {
                w[i][0] = *reinterpret_cast<const volatile uint32_t *>(from + 16 * kv_chunk(c.chunks, p.slot, j / 4) +
                                                                       4 * (j % 4));
            } else {
                const uint8_t *at = from + 16 * kv_chunk(c.chunks, p.slot, j / 2) + 8 * (j % 2);
                asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "l"(at));
            }
            word[i] = reinterpret_cast<const volatile uint32_t *>(head + 2 * c.page * c.row_bytes)[(is_v ? c.page : 0) +
                                                                                                   p.slot];
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int item = first + i * G;
            const bool is_v = item >= c.heads;
            if (item >= 2 * c.heads) continue;
            T *to = static_cast<T *>(const_cast<void *>(is_v ? a.v : a.k));
            if (!to) continue;
            const float s = __uint_as_float(U4 ? word[i] & 0xffff0000u : word[i]);
            const int z = U4 ? (int)(word[i] & 15u) : 128;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int q = U4 ? (int)(w[i][0] >> (4 * e) & 15u) : (int)(w[i][e / 4] >> (8 * (e % 4)) & 255u);
                x[e] = __fmul_rn((float)(q - z), s);
            }
            store8(to + row * (is_v ? a.ld_v : a.ld_k) + (int64_t)(item - (is_v ? c.heads : 0)) * c.D + d0, a.vec, x);
        }
    }
}

constexpr int kMaxKeep = 1024, kKeepThreads = 128;

struct KvKeepArgs {
    KvArgs c;
    const int32_t *keep, *n_keep;
    int ld_keep;
};

// A block has one sequence and 128 of its columns (16 bytes of a row, or the words, of a head's
// K or V); a thread moves its column of all kept tokens in order, which no other thread
// touches.  keep ascends, so keep[i] >= i: no source is a place that an earlier i has filled.
__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const __grid_constant__ KvKeepArgs a)
{
    const KvArgs &c = a.c;
    __shared__ int64_t from_page[kMaxKeep], to_page[kMaxKeep];
    __shared__ int slots[kMaxKeep];  // of both, 16 bits each
    const int b = blockIdx.y;
    grid_dependency_launch();
    grid_dependency_wait();
    const KvSeq s = kv_seq(c, b);
    const int n = *reinterpret_cast<const volatile int32_t *>(a.n_keep + b);
    const volatile int32_t *keep = a.keep + (int64_t)b * a.ld_keep;
    if (s.T < 0) return;
    bool bad = n < 0 || n > s.T || n > a.ld_keep;
    if (!bad)
        for (int i = threadIdx.x; i < n; i += kKeepThreads) {
            const int t = keep[i];
            bad = bad || t < 0 || t >= s.T || (i > 0 && keep[i - 1] >= t);
        }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) kv_bad(c);
        return;
    }
    for (int i = threadIdx.x; i < n; i += kKeepThreads) {
        const int64_t pf = (int64_t)s.len - s.T + keep[i], pt = (int64_t)s.len - s.T + i;
        from_page[i] = to_page[i] = -1;
        slots[i] = 0;
        if (pf == pt || pt < 0) continue;
        const int f = kv_page(c, b, (int)(pf / c.page)), t = kv_page(c, b, (int)(pt / c.page));
        if (f < 0 || t < 0) continue;
        from_page[i] = f * c.page_bytes;
        to_page[i] = t * c.page_bytes;
        slots[i] = (int)(pf % c.page) | (int)(pt % c.page) << 16;
    }
    __syncthreads();
    const int columns = 2 * (c.chunks + 1), col = blockIdx.x * kKeepThreads + threadIdx.x;
    if (col >= columns * c.heads) return;
    const int head = col / columns, x = col % columns, is_v = x / (c.chunks + 1), chunk = x % (c.chunks + 1);
    uint8_t *base = c.pages + (int64_t)head * c.head_bytes;
    auto move = [&](auto kind, auto at) {  // four at a time: loads, then stores
        using V = decltype(kind);
        for (int i0 = 0; i0 < n; i0 += 4) {
            V v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + e;
                if (i < n && from_page[i] >= 0)
                    v[e] = *reinterpret_cast<const V *>(base + from_page[i] + at(slots[i] & 0xffff));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + e;
                if (i < n && from_page[i] >= 0) *reinterpret_cast<V *>(base + to_page[i] + at(slots[i] >> 16)) = v[e];
            }
        }
    };
    if (chunk < c.chunks)
        move(uint4{}, [&](int slot) {
            return (is_v * c.page + slot) * c.row_bytes + 16 * kv_chunk(c.chunks, slot, chunk);
        });
    else
        move(uint32_t{}, [&](int slot) { return 2 * c.page * c.row_bytes + 4 * (is_v * c.page + slot); });
}

template <typename T, bool U4, int W>
qnn_status launch_io(KvIoArgs a, bool read, cudaStream_t s)
{
    const int per = kUnroll * (32 / W);
    a.parts = (2 * a.c.heads + per - 1) / per;
    const int64_t units = a.c.rows * a.parts, blocks = (units + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)sm_count() * 8));
    return read ? kv_launch(kv_read_kernel<T, U4, W>, grid, kWarps * 32, 0, s, a)
                : kv_launch(kv_write_kernel<T, U4, W>, grid, kWarps * 32, 0, s, a);
}

template <typename T, bool U4>
qnn_status launch_width(const KvIoArgs &a, bool read, cudaStream_t s)
{
    if (a.c.D <= 32) return launch_io<T, U4, 4>(a, read, s);
    if (a.c.D <= 64) return launch_io<T, U4, 8>(a, read, s);
    if (a.c.D <= 128) return launch_io<T, U4, 16>(a, read, s);
    return launch_io<T, U4, 32>(a, read, s);
}

template <typename T>
qnn_status launch_codes(const KvIoArgs &a, bool u4, bool read, cudaStream_t s)
{
    return u4 ? launch_width<T, true>(a, read, s) : launch_width<T, false>(a, read, s);
}

qnn_status kv_io(const void *k, const void *v, int x_dt, int64_t ld_k, int64_t ld_v, const qnn_kv_geom *g,
                 const qnn_kv_seqs *seqs, bool read, cudaStream_t s)
{
    KvIoArgs a = {};
    const qnn_status st = kv_args(g, seqs, &a.c);
    if (st != QNN_OK) return st;
    if (!is_float_dt(x_dt)) return QNN_ERR_UNSUPPORTED;
    const int64_t width = (int64_t)g->heads * g->D;
    a.ld_k = ld_k ? ld_k : width;
    a.ld_v = ld_v ? ld_v : width;
    const int64_t most = INT64_MAX / 8 / std::max<int64_t>(1, a.c.rows);
    if (a.ld_k < width || a.ld_v < width || a.ld_k > most || a.ld_v > most) return QNN_ERR_INVALID_ARG;
    if (a.c.batch == 0 || a.c.rows == 0) return QNN_OK;
    if (read ? !k && !v : !k || !v) return QNN_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return QNN_ERR_ALIGNMENT;
    a.k = k;
    a.v = v;
    a.vec = (a.ld_k * float_bytes(x_dt)) % 16 == 0 && (a.ld_v * float_bytes(x_dt)) % 16 == 0;
    if (!(a.c.status = status_word())) return QNN_ERR_CUDA;
    const bool u4 = g->kv_dt == QNN_U4;
    switch (x_dt) {
    case QNN_F32: return launch_codes<float>(a, u4, read, s);
    case QNN_F16: return launch_codes<__half>(a, u4, read, s);
    default: return launch_codes<__nv_bfloat16>(a, u4, read, s);
    }
}

}  // namespace
}  // namespace qnn

extern "C" size_t qnn_kv_page_bytes(const qnn_kv_geom *g)
{
    if (!qnn::kv_geom_ok(g)) return 0;
    return (size_t)g->heads * g->page * (2 * qnn::kv_row_bytes(*g) + 8);
}

extern "C" qnn_status q_kv_write(const void *k, const void *v, qnn_dtype x_dt, int64_t ld_k, int64_t ld_v,
                                 const qnn_kv_geom *g, const qnn_kv_seqs *seqs, qnn_stream_t stream)
{
    return qnn::kv_io(k, v, x_dt, ld_k, ld_v, g, seqs, false, (cudaStream_t)stream);
}

extern "C" qnn_status q_kv_read(void *k, void *v, qnn_dtype x_dt, int64_t ld_k, int64_t ld_v, const qnn_kv_geom *g,
                                const qnn_kv_seqs *seqs, qnn_stream_t stream)
{
    return qnn::kv_io(k, v, x_dt, ld_k, ld_v, g, seqs, true, (cudaStream_t)stream);
}

extern "C" qnn_status q_kv_keep(const qnn_kv_geom *g, const qnn_kv_seqs *seqs, const int32_t *keep, int64_t ld_keep,
                                const int32_t *n_keep, qnn_stream_t stream)
{
    qnn::KvKeepArgs a = {};
    const qnn_status st = qnn::kv_args(g, seqs, &a.c);
    if (st != QNN_OK) return st;
    if (ld_keep < 0) return QNN_ERR_INVALID_ARG;
    if (ld_keep > qnn::kMaxKeep) return QNN_ERR_UNSUPPORTED;
    if (a.c.batch == 0 || a.c.rows == 0 || ld_keep == 0) return QNN_OK;
    if (!keep || !n_keep) return QNN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(keep) & 3u) || (reinterpret_cast<uintptr_t>(n_keep) & 3u)) return QNN_ERR_ALIGNMENT;
    a.keep = keep;
    a.n_keep = n_keep;
    a.ld_keep = (int)ld_keep;
    if (!(a.c.status = qnn::status_word())) return QNN_ERR_CUDA;
    const int columns = 2 * (a.c.chunks + 1) * a.c.heads;
    const dim3 grid((unsigned)((columns + qnn::kKeepThreads - 1) / qnn::kKeepThreads), (unsigned)a.c.batch);
    return qnn::kv_launch(qnn::kv_keep_kernel, grid, qnn::kKeepThreads, 0, (cudaStream_t)stream, a);
}
