// qnn_kv.cu -- the cache of keys and values: quantised as it is written (q_kv_write), read
// back (q_kv_read), and its accepted tokens kept (q_kv_keep).
//
// All three move bytes.  A group of lanes, one for each 16 channels (8 for a read), has a token's head of K or
// V at a time: maxima by shuffles inside the group, one division for 1 / scale, and the rest by products that give
// what divisions give (so that codes are those of the definition, ties included).  A warp has
// some of the heads of a run of rows: it looks up the places of all of them at once, a lane a row (the
// chain of reads starts -> lens -> table is what a row costs), and has the next row's values on their
// way while it works on one.
//
// Bytes bound the read: 8 x 4096 tokens of 8 heads of 128, 8 bits to bf16, take 39 us, 5.2 TB/s.  A write is
// bound by latency and instructions: 4 sequences, 10 000 tokens in all, to 4 bits take 22 us, 20 million values (60
// with divisions for all values near ties); 16 x 4096 tokens of 8 heads of 128 written and read, 210 us in 8
// bits.  A warp has several rows at a time where a row has few heads (2 x 127238 tokens of one head of 64, fp32,
// written and read: 204 us with one, 79).  One token takes 5 us, latency.
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
    a->per16 = (uint32_t)g->page / 16;
    a->magic16 = (uint32_t)(((1ull << 32) + a->per16 - 1) / a->per16);
    a->status = nullptr;
    return QNN_OK;
}

namespace {

constexpr int kWarps = 8, kReadItems = 4;  // of a row, that a group of lanes reads at a time

struct KvIoArgs {
    KvArgs c;
    const void *k, *v;
    int64_t ld_k, ld_v;
    int run;    // rows of a warp; their places are looked up together, one by a lane
    int log_r;  // 2^log_r groups of lanes have a row, each a head of K or V; the warp's others the next rows
    int vec;    // rows of k and v start on 16-byte boundaries
};

// The place of a row: its position's page and offset in it; page -1: none.
struct Place {
    int page, slot;  // slot: the token in the page
    int seq;         // 0: no sequence has the row
};

// The sequence whose rows hold `row`: the number of starts[1 .. batch] that are <= row.
// (Where they descend the answer is some sequence, and what follows is checked.)
__device__ __forceinline__ int seq_of_row(const KvArgs &a, int row)
{
    if (!a.starts) return (unsigned)row / (unsigned)a.tokens;
    int lo = 0, n = a.batch;  // the answer is in lo .. lo + n
    const volatile int32_t *st = a.starts + 1;
#pragma unroll 1
    while (n > 0) {
        const int half = n >> 1;
        if (st[lo + half] <= row) lo += half + 1, n -= half + 1;
        else n = half;
    }
    return lo;
}

__device__ __forceinline__ Place place_of(const KvArgs &a, int row)
{
    Place p = {-1, 0, 0};
    if (row >= a.rows) return p;
    const int b = seq_of_row(a, row);
    if (b >= a.batch) return p;
    const KvSeq s = kv_seq(a, b);
    const int t = row - (int)s.first;
    if (s.T < 0 || t < 0 || t >= s.T) return p;
    p.seq = 1;
    const int pos = s.len - s.T + t;
    if (pos < 0) return p;
    int tile;
    const int index = kv_page_index(a, pos >> 4, &tile);
    p.page = kv_page(a, b, index);
    p.slot = tile * 16 + (pos & 15);
    return p;
}

// Eight values as they lie in memory.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, int vec, Raw8<T> &x)
{
    if (vec) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.w[i].x), "=r"(x.w[i].y), "=r"(x.w[i].z), "=r"(x.w[i].w)
                         : "l"(reinterpret_cast<const uint4 *>(p) + i));
        }
    } else {
        T *e = reinterpret_cast<T *>(x.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = p[i];
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

// W lanes have an item's channels; `live`: this lane has some.
template <int W>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int d = W / 2; d > 0; d /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// a / b, rounded to nearest as by a division, where b has 8 significant bits at most, `per` is 1 / b rounded, and
// nothing underflows: a product, what it leaves, and the product corrected by that (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  The corrected value before its rounding is
// within 2^-45 of a / b, relatively.  a / b is no middle of two fp32 numbers (b times one, which has 25 bits and is
// odd, has more than 24), and so lies 2^-33 or more from each: both round to the same.
__device__ __forceinline__ float2 quotients(float2 a, float2 b, float2 per)
{
    const float2 q = mul2(a, per);
    return fma2(fma2(make_float2(-q.x, -q.y), b, a), per, q);
}

template <typename T, bool U4, int W>
__global__ void __launch_bounds__(kWarps * 32, 3) kv_write_kernel(const __grid_constant__ KvIoArgs a)
{
    const KvArgs &c = a.c;
    constexpr int G = 32 / W;  // groups of a warp
    const int lane = threadIdx.x & 31, group = lane / W, j = lane % W, d0 = 16 * j;
    const int per = G >> a.log_r, sub = group >> a.log_r;  // rows at a time
    const bool live = d0 < c.D;
    grid_dependency_launch();
    grid_dependency_wait();
    const int64_t r0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * a.run;
    const int rows = (int)min((int64_t)a.run, c.rows - r0);
    if (rows <= 0) return;
    const int item = (blockIdx.y << a.log_r) + (group & ((1 << a.log_r) - 1));  // K's heads, then V's
    const bool is_v = item >= c.heads, some = item < 2 * c.heads && live;
    const int64_t pitch = is_v ? a.ld_v : a.ld_k;
    const T *from = static_cast<const T *>(is_v ? a.v : a.k) + (r0 + sub) * pitch +
                    (int64_t)(item - (is_v ? c.heads : 0)) * c.D + d0;
    // Rows on their way, as they lie in memory, and converted when their turn comes: two, or one of fp32, whose
    // second would not fit the registers (prompts written and read in 4 bits: 42 us, 48 with one).
    constexpr int kAhead = sizeof(T) == 2 ? 2 : 1;
    Raw8<T> ahead[kAhead][2];
    auto ask = [&](int t, Raw8<T> (&to)[2]) {
        if (some && t + sub < rows) {
            load8(from + t * pitch, a.vec, to[0]);
            load8(from + t * pitch + 8, a.vec, to[1]);
        } else {
#pragma unroll
            for (int e = 0; e < (int)sizeof(T) / 2; ++e) to[0].w[e] = to[1].w[e] = make_uint4(0, 0, 0, 0);
        }
    };
    ask(0, ahead[0]);
    if (kAhead > 1) ask(per, ahead[kAhead - 1]);
    const Place places = place_of(c, lane < rows ? (int)r0 + lane : INT32_MAX);
#pragma unroll 1
    for (int t = 0; t < rows; t += per) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const T *raw = reinterpret_cast<const T *>(ahead[0][i].w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * i + e] = to_f32(raw[e]);
            if constexpr (kAhead > 1) ahead[0][i] = ahead[1][i];
        }
        ask(t + kAhead * per, ahead[kAhead - 1]);
        Place p;  // of no row: that of a lane without one, -1
        p.page = __shfl_sync(0xffffffffu, places.page, t + sub);
        p.slot = __shfl_sync(0xffffffffu, places.slot, t + sub);
        if (__all_sync(0xffffffffu, p.page < 0)) continue;
        uint8_t *base = c.pages + p.page * c.page_bytes;
        float hi = 0.0f, lo = 0.0f;  // the largest value and -min, both 0 at least (NaN aside)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            hi = U4 ? max3(hi, x[e], x[e + 1]) : max3(hi, fabsf(x[e]), fabsf(x[e + 1]));
            if (U4) lo = max3(lo, -x[e], -x[e + 1]);
        }
        if (U4) lo = group_max<W>(lo);
        hi = group_max<W>(hi);
        if (__any_sync(0xffffffffu, fmaxf(hi, lo) == INFINITY)) {  // once more, of what is finite
            hi = lo = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (!finite(x[e])) continue;
                hi = fmaxf(hi, U4 ? x[e] : fabsf(x[e]));
                if (U4) lo = fmaxf(lo, -x[e]);
            }
            hi = group_max<W>(hi);
            if (U4) lo = group_max<W>(lo);
        }
        float s, z = 0.0f;
        uint32_t q[16];
        constexpr float kInteger = 12582912.0f;  // 1.5 * 2^23: a sum with it is an integer in the low bits
        bool plain = fmaxf(hi, lo) > 0x1p-60f;
        if constexpr (U4) {
            const float2 of = quotients(make_float2(hi, lo), both(15.0f), both(1.0f / 15.0f));
            s = __bfloat162float(__float2bfloat16_rn(__fadd_rn(of.x, of.y)));
            const float2 by = both(s), per = both(__fdiv_rn(1.0f, s));
            z = fminf(rintf(quotients(both(lo), by, per).x), 15.0f);
            float2 sum = both(0.0f);  // not a number where a value is none, or infinite
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float2 t = quotients(make_float2(x[e], x[e + 1]), by, per);
                sum = add2(sum, t);
                const float2 r = add2(add2(t, both(kInteger)), both(z));
                q[e] = __float_as_uint(fminf(fmaxf(r.x, kInteger), kInteger + 15.0f));
                q[e + 1] = __float_as_uint(fminf(fmaxf(r.y, kInteger), kInteger + 15.0f));
            }
            plain = plain && sum.x + sum.y == sum.x + sum.y;
        } else {
            s = quotients(both(hi), both(127.0f), both(1.0f / 127.0f)).x;
            // By a product with 1 / s: that is within 2^-21 of the quotient, relatively, and so the same integer
            // but near a tie.
            const float2 per = both(__fdiv_rn(1.0f, s));
            float far = 0.0f;  // from the nearest integer
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float2 t = mul2(make_float2(x[e], x[e + 1]), per), r = add2(t, both(kInteger));
                const float2 d = add2(add2(r, both(-kInteger)), make_float2(-t.x, -t.y));
                // NaN does not pass the comparison: max would drop it
                far = max3(far, fabsf(d.x) < 0.4999f ? 0.0f : 1.0f, fabsf(d.y) < 0.4999f ? 0.0f : 1.0f);
                q[e] = __float_as_uint(r.x), q[e + 1] = __float_as_uint(r.y);
            }
            plain = plain && far == 0.0f;
        }
        if (!plain) {  // by division
            if constexpr (U4) {
                s = __bfloat162float(__float2bfloat16_rn(__fadd_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f))));
                z = s > 0.0f ? fminf(rintf(__fdiv_rn(lo, s)), 15.0f) : 0.0f;
            } else {
                s = __fdiv_rn(hi, 127.0f);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float v = x[e], r = s > 0.0f && v == v ? rintf(__fdiv_rn(v, s)) : 0.0f;
                q[e] = U4 ? (uint32_t)fminf(fmaxf(__fadd_rn(r, z), 0.0f), 15.0f)
                          : (uint32_t)(int)fminf(fmaxf(r, -127.0f), 127.0f);
            }
        }
        // the low bytes of all
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = prmt(prmt(q[4 * e], q[4 * e + 1], 0x0040), prmt(q[4 * e + 2], q[4 * e + 3], 0x0040), 0x5410);
        if (!some || p.page < 0) continue;
        uint8_t *head = base + (int64_t)(item - (is_v ? c.heads : 0)) * c.head_bytes;
        uint8_t *to = head + (is_v ? c.page * c.row_bytes : 0) + p.slot * c.row_bytes;
        if constexpr (U4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] |= w[e] >> 4;  // bytes 0 and 2: two codes each
            *reinterpret_cast<uint2 *>(to + 16 * kv_chunk(c.chunks, p.slot, j / 2) + 8 * (j % 2)) =
                make_uint2(prmt(w[0], w[1], 0x6420), prmt(w[2], w[3], 0x6420));
        } else {
            *reinterpret_cast<uint4 *>(to + 16 * kv_chunk(c.chunks, p.slot, j)) =
                make_uint4(w[0] ^ 0x80808080u, w[1] ^ 0x80808080u, w[2] ^ 0x80808080u, w[3] ^ 0x80808080u);
        }
        if (j == 0) {
            const uint32_t word = U4 ? __float_as_uint(s) | (uint32_t)z : __float_as_uint(s);
            reinterpret_cast<uint32_t *>(head + 2 * c.page * c.row_bytes)[(is_v ? c.page : 0) + p.slot] = word;
        }
    }
}

// Blocks of an SM: four want 64 registers, which 8 bits to 16-bit values nearly do with (8 x 4096 tokens: 39 us, 43
// with three), fp32 does not (10575 tokens: 36 us, 27 with three).
template <typename T, bool U4, int W>
__global__ void __launch_bounds__(kWarps * 32, U4 || sizeof(T) == 4 ? 3 : 4) kv_read_kernel(const __grid_constant__ KvIoArgs a)
{
    const KvArgs &c = a.c;
    constexpr int G = 32 / W;
    const int lane = threadIdx.x & 31, group = lane / W, j = lane % W, d0 = 8 * j;
    const int per = G >> a.log_r, sub = group >> a.log_r, next = 1 << a.log_r;  // rows at a time; from head to head
    const bool live = d0 < c.D;
    grid_dependency_launch();
    grid_dependency_wait();
    const int first = blockIdx.y * kReadItems * next + (group & (next - 1));
    const int64_t r0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * a.run;
    const int rows = (int)min((int64_t)a.run, c.rows - r0);
    if (rows <= 0) return;
    const Place places = place_of(c, lane < rows ? (int)r0 + lane : INT32_MAX);
    uint32_t ahead[kReadItems][2], ahead_word[kReadItems];
    auto ask = [&](int t) {
        const int page = __shfl_sync(0xffffffffu, places.page, t + sub), slot = __shfl_sync(0xffffffffu, places.slot, t + sub);
#pragma unroll
        for (int i = 0; i < kReadItems; ++i) {
            const int item = first + i * next;
            const bool is_v = item >= c.heads;
            ahead[i][0] = ahead[i][1] = U4 ? 0 : 0x80808080u;
            ahead_word[i] = 0;
            if (item >= 2 * c.heads || page < 0 || !live) continue;
            const uint8_t *head = c.pages + page * c.page_bytes + (int64_t)(item - (is_v ? c.heads : 0)) * c.head_bytes;
            const uint8_t *from = head + (is_v ? c.page * c.row_bytes : 0) + slot * c.row_bytes;
            if constexpr (U4) {
                ahead[i][0] = *reinterpret_cast<const volatile uint32_t *>(from + 16 * kv_chunk(c.chunks, slot, j / 4) +
                                                                           4 * (j % 4));
            } else {
                const uint8_t *at = from + 16 * kv_chunk(c.chunks, slot, j / 2) + 8 * (j % 2);
                asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(ahead[i][0]), "=r"(ahead[i][1]) : "l"(at));
            }
            ahead_word[i] =
                reinterpret_cast<const volatile uint32_t *>(head + 2 * c.page * c.row_bytes)[(is_v ? c.page : 0) + slot];
        }
    };
    ask(0);
#pragma unroll 1
    for (int t = 0; t < rows; t += per) {
        const int64_t r = r0 + t + sub;
        const int seq = __shfl_sync(0xffffffffu, places.seq, t + sub);
        uint32_t w[kReadItems][2], word[kReadItems];
#pragma unroll
        for (int i = 0; i < kReadItems; ++i) w[i][0] = ahead[i][0], w[i][1] = ahead[i][1], word[i] = ahead_word[i];
        if (t + per < rows) ask(t + per);
        if (!seq || !live) continue;
#pragma unroll
        for (int i = 0; i < kReadItems; ++i) {
            const int item = first + i * next;
            const bool is_v = item >= c.heads;
            if (item >= 2 * c.heads) continue;
            T *to = static_cast<T *>(const_cast<void *>(is_v ? a.v : a.k));
            if (!to) continue;
            const float s = __uint_as_float(U4 ? word[i] & 0xffff0000u : word[i]);
            // 2^23 + a code, by its bits, less 2^23 and the zero point
            const float2 less = both(-8388608.0f - (U4 ? (float)(word[i] & 15u) : 128.0f));
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float2 v;
                if constexpr (U4) {
                    v = make_float2(__uint_as_float((w[i][0] >> (4 * e) & 15u) | 0x4b000000u),
                                    __uint_as_float((w[i][0] >> (4 * e + 4) & 15u) | 0x4b000000u));
                } else {
                    v = make_float2(__uint_as_float(prmt(w[i][e / 4], 0x4b000000u, 0x7440 + e % 4)),
                                    __uint_as_float(prmt(w[i][e / 4], 0x4b000000u, 0x7441 + e % 4)));
                }
                v = mul2(add2(v, less), both(s));
                x[e] = v.x, x[e + 1] = v.y;
            }
            store8(to + r * (is_v ? a.ld_v : a.ld_k) + (int64_t)(item - (is_v ? c.heads : 0)) * c.D + d0, a.vec, x);
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
// Latency bounds it (8 tokens' loads at a time): 32 sequences, 64 drafted tokens of 8 heads of 128 each, 8 us.
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
        const int pf = s.len - s.T + keep[i], pt = s.len - s.T + i;
        from_page[i] = to_page[i] = -1;
        slots[i] = 0;
        if (pf == pt || pt < 0) continue;
        int tile_f, tile_t;
        const int index_f = kv_page_index(c, pf >> 4, &tile_f), index_t = kv_page_index(c, pt >> 4, &tile_t);
        const int f = kv_page(c, b, index_f), t = kv_page(c, b, index_t);
        if (f < 0 || t < 0) continue;
        from_page[i] = f * c.page_bytes;
        to_page[i] = t * c.page_bytes;
        slots[i] = (tile_f * 16 + (pf & 15)) | (tile_t * 16 + (pt & 15)) << 16;
    }
    __syncthreads();
    const int columns = 2 * (c.chunks + 1), col = blockIdx.x * kKeepThreads + threadIdx.x;
    if (col >= columns * c.heads) return;
    const int head = col / columns, x = col % columns, is_v = x / (c.chunks + 1), chunk = x % (c.chunks + 1);
    uint8_t *base = c.pages + (int64_t)head * c.head_bytes;
    constexpr int kAtOnce = 8;
    auto move = [&](auto kind, auto at) {  // some at a time: loads, then stores
        using V = decltype(kind);
        for (int i0 = 0; i0 < n; i0 += kAtOnce) {
            V v[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const int i = i0 + e;
                if (i < n && from_page[i] >= 0)
                    v[e] = *reinterpret_cast<const V *>(base + from_page[i] + at(slots[i] & 0xffff));
            }
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
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
    // A warp's groups have the heads of one row or, where those are fewer, of several.  Where they are more there
    // is a row of blocks for each part of them.
    const int groups = 32 / (read ? W : W / 2);
    a.log_r = 0;
    while (1 << a.log_r < std::min(groups, 2 * a.c.heads)) ++a.log_r;
    const int per = groups >> a.log_r, items = (read ? kReadItems : 1) << a.log_r;
    const int parts = (2 * a.c.heads + items - 1) / items;
    // Rows of a warp: as many as let all warps run at once, 32 at most, and for a read 8 turns, whose later blocks
    // even out the rest (8 x 4096 tokens of 8 heads of 128 in 8 bits to bf16: 38 us, 49 with 32).
    const int64_t turns = (a.c.rows * parts / per + sm_count() * 24 - 1) / (sm_count() * 24);
    a.run = (int)std::min<int64_t>(32, std::min<int64_t>(read ? 8 : 32, std::max<int64_t>(1, turns)) * per);
    const int64_t block_rows = (int64_t)kWarps * a.run;
    const dim3 grid((unsigned)((a.c.rows + block_rows - 1) / block_rows), (unsigned)parts);
    return read ? kv_launch(kv_read_kernel<T, U4, W>, grid, kWarps * 32, 0, s, a)
                : kv_launch(kv_write_kernel<T, U4, W / 2>, grid, kWarps * 32, 0, s, a);
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
