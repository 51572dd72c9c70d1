// qnn_kv_attn_few.cu -- q_kv_attn for few rows of a head of the cache (up to 16 at a time: the
// heads of q that share it, times the newest tokens): decoding; of more than 128 channels up to 32, in large
// batches all.
//
//   S^T = K Q^T,  P^T = e^(S^T - m),  O^T = V^T P^T
// on mma.sync m16n8k16 with the codes as the A operand (16 tokens, or 16 channels) and 8 rows as
// N: codes go from shared memory to A fragments in registers, no value twice, and P^T's fragment
// is S^T's transposed 8 x 8 by 8 x 8 (movmatrix).  A code becomes an f16 integer, its zero point taken off, by a
// magic number and one subtraction; the products are exact, scales of K multiply the scores, scales of V the
// weights.  (Codes as they are stored, as f16 numbers u 2^-24, and zero points off the sums, are 5% faster in 4
// bits; but a product's unit then is its number's exponent, 2^-14, and sums lose ten bits.)
//
// The stream of codes is what it cannot do without: 64 sequences of 8192 tokens, 8 of 64 heads, in 8 bits take
// 141 us, 4.4 TB/s; the copies alone take 109, the rest alone 113, and a warp of each scheduler's four waits
// for memory, another for its chain of products.  One sequence of 131072 tokens in 4 bits: 56 us, 2.5 TB/s, by
// instructions (450 for a tile of 16 tokens).  Each warp has a ring of its own in shared memory, stages
// of 16 tokens (their K and V rows and words), filled by asynchronous copies; warps meet only
// where an item ends.  Maxima move only when a score passes the warp's by 2^8 (the
// weights have that room), which one vote a tile finds.
#include <type_traits>
#include "qnn_kv_attn.cuh"

namespace qnn {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
static_assert(kAttnChunk == 16 * kWarps, "a unit is a tile for each warp");

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

// N words from shared memory, aligned to their size (16 bytes at most at a time)
template <int N>
__device__ __forceinline__ void lds(uint32_t at, uint32_t *w)
{
    if constexpr (N == 1) w[0] = lds32(at);
    else if constexpr (N == 2) {
        const uint2 v = lds64(at);
        w[0] = v.x, w[1] = v.y;
    } else {
        const uint4 v = lds_v4(at);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
}

// DP: channels, D rounded up to 64, 128 or 256.  NT: tiles of 8 rows.
template <bool U4, int DP, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kChunks = DP / (U4 ? 32 : 16);   // of a row, at most
    static constexpr int kKWords = DP / (U4 ? 32 : 16);   // of a token's K that a lane has
    static constexpr int kVWords = DP / (U4 ? 64 : 32);   // of a token's V
    static constexpr int kSteps = DP / 16;                // of K, and tiles of 16 channels of V
    static constexpr bool kQRegs = NT * DP <= 256;        // q's fragments in registers
    static constexpr int kMinBlocks = NT * DP <= 128 ? 2 : 1;
    static constexpr int kPitch = DP + 4;                 // of a row where warps join
};

// The chunk, and the byte in it, at which a lane's words from w on begin: K's words of lane j (0..3),
// V's of lane g (0..7).
template <bool U4, int DP>
__device__ __forceinline__ int k_chunk(int j, int w) { return U4 && DP == 64 ? j / 2 : 4 * (w / 4) + j; }
template <bool U4, int DP>
__device__ __forceinline__ int k_byte(int j) { return U4 && DP == 64 ? 8 * (j % 2) : 0; }
template <bool U4, int DP>
__device__ __forceinline__ int v_byte(int g)  // in the row, before the order of chunks
{
    constexpr int bytes = U4 ? DP / 16 : DP == 64 ? 8 : 16;
    return bytes * g;
}

// Channel of value e of the lane's words of K (in fragment order: two for each register), and of
// element (tile i, half) of the sums.
template <bool U4, int DP>
__device__ __forceinline__ int k_channel(int j, int step, int e)  // e: k = 2j, 2j+1, 2j+8, 2j+9
{
    if constexpr (U4) {
        const int w = step / 2, n = (step % 2) * 2 + (e / 2) + 4 * (e % 2);  // nibbles n, n + 4
        if (DP == 64) return 16 * j + 8 * w + n;
        return 128 * (w / 4) + 32 * j + 8 * (w % 4) + n;
    } else {
        return 64 * (step / 4) + 16 * j + 4 * (step % 4) + e;
    }
}
template <bool U4, int DP>
__device__ __forceinline__ int sum_channel(int g, int i, int half)
{
    if constexpr (U4) return DP / 8 * g + 2 * i + half;
    else return DP == 64 ? 8 * g + 2 * i + half : 128 * (i / 8) + 16 * g + 2 * (i % 8) + half;
}

// Finding an item is kept out of the loop from tile to tile, which has to stay in the instruction cache.
__device__ __noinline__ AttnCursor find(const KvAttnArgs &a, const int64_t *sums, int64_t x, int width)
{
    return attn_find(a, sums, x, width);
}
__device__ __noinline__ AttnCursor next_rows(const KvAttnArgs &a, AttnCursor c, int width)
{
    return attn_next_rows(a, c, width);
}
__device__ __forceinline__ void next(const KvAttnArgs &a, AttnCursor &c, int width)
{
    if (++c.chunk < c.units) return;
    c.chunk = 0;
    if (++c.h >= a.c.heads) c = next_rows(a, c, width);
}

// A stage: K rows, V rows, K words, V words of 16 tokens.
__host__ __device__ inline int stage_bytes(int row_bytes) { return 16 * (2 * row_bytes + 8); }

template <bool U4, int DP, int NT>
__global__ void __launch_bounds__(kThreads, Shape<U4, DP, NT>::kMinBlocks)
kv_attn_few_kernel(const __grid_constant__ KvAttnArgs a)
{
    using S = Shape<U4, DP, NT>;
    const KvArgs &c = a.c;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float4 stats[kWarps][S::kRows];    // maximum, unit of V's scales, sum of weights
    __shared__ float row_unit[kWarps][S::kRows];  // where they are apart
    __shared__ uint2 q_smem[S::kQRegs ? 1 : NT * S::kSteps * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
    const int stage_b = stage_bytes(c.row_bytes), ST = a.stages;
    float *join = reinterpret_cast<float *>(smem);  // [warps][8][kPitch]
    uint8_t *ring = smem + kWarps * 8 * S::kPitch * 4 + warp * ST * stage_b;
    int64_t *sums = reinterpret_cast<int64_t *>(smem + kWarps * (8 * S::kPitch * 4 + ST * stage_b) + 128);
    const uint32_t ring_at = smem_u32(ring);

    grid_dependency_launch();
    grid_dependency_wait();
    const AttnShare share(attn_sums<kThreads>(a, sums, S::kRows), a.blocks, blockIdx.x);
    if (share.from >= share.to) {
        if (threadIdx.x == 0) attn_record(a, -1, 0, 0, 0, 0);
        return;
    }

    // the copies' side: `ahead` is the unit whose page has been looked up
    AttnCursor ahead = find(a, sums, share.from, S::kRows), at = ahead;
    int64_t unasked = share.to - share.from;  // units whose copies are still to be issued
    int entry = 0, in_page = 0;
    bool some = false;
    auto look_up = [&]() {  // what it asks for is looked at a tile later
        const int tile = ahead.chunk * kWarps + warp;
        some = tile * 16 < ahead.len;
        if (some) entry = kv_entry(c, ahead.b, kv_page_index(c, tile, &in_page));
    };
    uint32_t absent = 0;  // stages whose tile is not there; kApart: the rows' units are in row_unit
    constexpr uint32_t kApart = 1u << 31;
    auto ask = [&](int stage) {  // a group of copies, if only an empty one
        if (unasked > 0) {
            const int page = some ? kv_checked(c, entry) : -1;
            const bool there = page >= 0;
            absent = there ? absent & ~(1u << stage) : absent | 1u << stage;
            if (there) {
                const uint32_t to = ring_at + stage * stage_b + 16 * lane;
                const uint8_t *head = c.pages + page * c.page_bytes + (int64_t)ahead.h * c.head_bytes;
                const int rows = 16 * c.row_bytes, all = c.page * c.row_bytes;
                const uint8_t *k = head + in_page * rows + 16 * lane;
#pragma unroll
                for (int e = 0; e < 16 * S::kChunks; e += 32)
                    if (e + lane < 16 * c.chunks) {
                        copy_async16(to + 16 * e, k + 16 * e);
                        copy_async16(to + rows + 16 * e, k + all + 16 * e);
                    }
                if (lane < 8)
                    copy_async16(to + 2 * rows, head + 2 * all + (lane < 4 ? 0 : 4 * c.page - 64) + in_page * 64 + 16 * lane);
            }
            if (--unasked > 0) {
                next(a, ahead, S::kRows);
                look_up();
            }
        }
        copies_commit();
    };
    look_up();
    for (int i = 0; i < ST; ++i) ask(i);

    // where a lane's words are in a stage: of K's token g, of V's tokens 2j and 2j + 1 (8 tokens on: the same
    // order of chunks, 8 rows on)
    constexpr int kKLoads = (S::kKWords + 3) / 4, kVLoads = (S::kVWords + 3) / 4;
    int k_off[kKLoads], v_off[2][kVLoads];
#pragma unroll
    for (int w = 0; w < kKLoads; ++w)
        k_off[w] = g * c.row_bytes + 16 * kv_chunk(c.chunks, g, k_chunk<U4, DP>(j, 4 * w)) + k_byte<U4, DP>(j);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 0; w < kVLoads; ++w) {
            const int byte = v_byte<U4, DP>(g) + w * 128;
            v_off[e][w] = (16 + 2 * j + e) * c.row_bytes + 16 * kv_chunk(c.chunks, 2 * j + e, byte / 16) + byte % 16;
        }
    const int eight = 8 * c.row_bytes;

    int stage = 0;
    int64_t x = share.from;
    while (x < share.to) {
        // one item, or the part of it that is this block's
        const int64_t item_first = x - at.chunk;  // its place in the line
        const int64_t item_end = item_first + at.units, end = min(item_end, share.to), first = at.first;
        const int row0 = at.rt * S::kRows, head = at.h;
        const int width = (int)min((int64_t)S::kRows, (int64_t)at.T * a.group - row0);
        const int t_first = row0 / a.group, t_last = (row0 + width - 1) / a.group;
        const bool starts_here = item_first >= share.from, ends_here = item_end <= share.to;
        if (threadIdx.x == 0 && end == share.to)
            attn_record(a, starts_here && !ends_here ? share.block_of(item_end - 1) : -1, first, row0, width, head);

        // q's fragments: B of m16n8k16, column g, each row scaled to f16's range
        uint32_t qf[S::kQRegs ? NT : 1][S::kQRegs ? S::kSteps : 1][2];
        float cq[NT][2];  // of rows 2j, 2j + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = row0 + 8 * nt + g;
            const bool live = 8 * nt + g < width;
            const int64_t qat = (first + r / a.group) * a.ld_q + (int64_t)(head * a.group + r % a.group) * c.D;
            const uint16_t *qp = static_cast<const uint16_t *>(a.q) + qat;
            if (S::kQRegs || warp == nt % kWarps) {
                float top = 0.0f;
                float v[S::kSteps][4];
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int d = k_channel<U4, DP>(j, s, e);
                        uint16_t raw = 0;
                        if (live && d < c.D) asm volatile("ld.global.u16 %0, [%1];" : "=h"(raw) : "l"(qp + d));
                        v[s][e] = a.bf16 ? __uint_as_float((uint32_t)raw << 16) : __half2float(__ushort_as_half(raw));
                        top = fmaxf(top, fabsf(v[s][e]));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const RowUnit by(top);
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s) {
                    const __half2 lo = __floats2half2_rn(by.up(v[s][0]), by.up(v[s][1]));
                    const __half2 hi = __floats2half2_rn(by.up(v[s][2]), by.up(v[s][3]));
                    const uint32_t b0 = *reinterpret_cast<const uint32_t *>(&lo);
                    const uint32_t b1 = *reinterpret_cast<const uint32_t *>(&hi);
                    if constexpr (S::kQRegs) qf[nt][s][0] = b0, qf[nt][s][1] = b1;
                    else q_smem[(nt * S::kSteps + s) * 32 + lane] = make_uint2(b0, b1);
                }
                if constexpr (S::kQRegs) {
                    cq[nt][0] = __shfl_sync(0xffffffffu, by.down, 8 * j);
                    cq[nt][1] = __shfl_sync(0xffffffffu, by.down, 8 * j + 4);
                } else if (j == 0) {
                    stats[0][8 * nt + g].x = by.down;
                }
            }
        }
        if constexpr (!S::kQRegs) {
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) cq[nt][0] = stats[0][8 * nt + 2 * j].x, cq[nt][1] = stats[0][8 * nt + 2 * j + 1].x;
            __syncthreads();
        }

        float acc[NT][S::kSteps][4], m[NT][2], ref[NT][2], l[NT][2];
        float per_unit = pow2i(126);  // V's scales are taken in units of 2^k
        absent &= ~kApart;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][s][e] = 0.0f;
            m[nt][0] = m[nt][1] = -INFINITY;
            ref[nt][0] = ref[nt][1] = l[nt][0] = l[nt][1] = 0.0f;
        }

        const int seen_by_all = a.mask ? at.len - at.T : min(at.len, at.len - at.T + t_first + 1);
        const int seen_by_any = a.mask ? at.len : at.len - at.T + t_last + 1;
        int pos0 = (at.chunk * kWarps + warp) * 16;
        // The tiles of which every row sees all, then the others: a loop each, so that the first, where nearly all
        // tiles are, is no longer than it must be.
        auto tiles = [&](auto kind, int left) {
            constexpr bool whole = decltype(kind)::value;
#pragma unroll 1
            for (; left > 0; --left) {
                copies_wait(ST - 1);
                __syncwarp();
                if (!(absent >> stage & 1u) && (whole || pos0 < seen_by_any)) {
                    const uint32_t k_at = ring_at + stage * stage_b, w_at = k_at + 4 * eight;
                    // scales of K and V of tokens g and g + 8
                    const uint32_t wk0 = lds32(w_at + 4 * g), wk1 = lds32(w_at + 4 * g + 32);
                    const uint32_t wv0 = lds32(w_at + 64 + 4 * g), wv1 = lds32(w_at + 64 + 4 * g + 32);
                    float s[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
                    {
                        uint32_t k0[S::kKWords], k1[S::kKWords];
                        constexpr int step_w = S::kKWords < 4 ? S::kKWords : 4;
#pragma unroll
                        for (int w = 0; w < S::kKWords; w += step_w) {
                            lds<step_w>(k_at + k_off[w / 4], k0 + w);
                            lds<step_w>(k_at + k_off[w / 4] + eight, k1 + w);
                        }
                        const Zero z0 = zero_of(wk0 & 15u, wk0 & 15u), z1 = zero_of(wk1 & 15u, wk1 & 15u);
#pragma unroll
                        for (int w = 0; w < S::kKWords; ++w) {
                            uint32_t f[U4 ? 2 : 1][4];
                            if constexpr (U4) {
                                uint32_t r0[4], r1[4];
                                u4_pairs(k0[w], z0, r0);
                                u4_pairs(k1[w], z1, r1);
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    f[e][0] = r0[2 * e], f[e][1] = r1[2 * e], f[e][2] = r0[2 * e + 1], f[e][3] = r1[2 * e + 1];
                                }
                            } else {
                                s8_pairs(k0[w], f[0][0], f[0][2]);
                                s8_pairs(k1[w], f[0][1], f[0][3]);
                            }
#pragma unroll
                            for (int e = 0; e < (U4 ? 2 : 1); ++e) {
                                const int st = w * (U4 ? 2 : 1) + e;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    if constexpr (S::kQRegs) mma16816(s[nt], f[e], qf[nt][st][0], qf[nt][st][1]);
                                    else {
                                        const uint2 b = q_smem[(nt * S::kSteps + st) * 32 + lane];
                                        mma16816(s[nt], f[e], b.x, b.y);
                                    }
                                }
                            }
                        }
                    }
                    // scores in units of log2; s[.][0, 1]: token g, rows 2j, 2j + 1; [2, 3]: token g + 8
                    const float sk0 = __uint_as_float(U4 ? wk0 & 0xffff0000u : wk0) * a.scale_log2;
                    const float sk1 = __uint_as_float(U4 ? wk1 & 0xffff0000u : wk1) * a.scale_log2;
                    float sv0 = __uint_as_float(U4 ? wv0 & 0xffff0000u : wv0);
                    float sv1 = __uint_as_float(U4 ? wv1 & 0xffff0000u : wv1);
                    bool over = false;
                    if constexpr (!whole) {  // words beyond the sequence hold anything
                        if (pos0 + g >= at.len) sv0 = 0.0f;
                        if (pos0 + g + 8 >= at.len) sv1 = 0.0f;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        s[nt][0] = s[nt][0] * (cq[nt][0] * sk0), s[nt][1] = s[nt][1] * (cq[nt][1] * sk0);
                        s[nt][2] = s[nt][2] * (cq[nt][0] * sk1), s[nt][3] = s[nt][3] * (cq[nt][1] * sk1);
                        if constexpr (!whole) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int t = min((row0 + 8 * nt + 2 * j + (e & 1)) / a.group, at.T - 1);
                                if (!attn_sees(a, at, t, pos0 + g + 8 * (e >> 1))) s[nt][e] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) over = over || fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + kAttnSlack;
                    }
                    float w0 = sv0 * per_unit, w1 = sv1 * per_unit;
                    over = over || w0 > 1.0f || w1 > 1.0f;
                    if (__any_sync(0xffffffffu, over)) {
                        // new maxima of rows 2j, 2j + 1 (over the lanes of all tokens); a new unit, of the tokens that
                        // all rows see, or one for each row
                        const uint32_t su = max(whole || pos0 + g < seen_by_all ? __float_as_uint(sv0) : 0u,
                                                whole || pos0 + g + 8 < seen_by_all ? __float_as_uint(sv1) : 0u);
                        const float before = pow2_inverse(per_unit);
                        per_unit = pow2_inverse(fmaxf(before, pow2_above(__uint_as_float(__reduce_max_sync(0xffffffffu, su)))));
                        const float ratio = before * per_unit;
                        w0 = sv0 * per_unit, w1 = sv1 * per_unit;
                        bool apart = false, each = false;
                        if constexpr (!whole) {
                            apart = absent & kApart;
                            each = apart || __any_sync(0xffffffffu, w0 > 1.0f || w1 > 1.0f);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float f[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float v = fmaxf(s[nt][e], s[nt][e + 2]);
#pragma unroll
                                for (int d = 4; d < 32; d *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                                const float top = fmaxf(m[nt][e], v);
                                f[e] = m[nt][e] == -INFINITY ? 0.0f : ex2(m[nt][e] - top);
                                m[nt][e] = top;
                                ref[nt][e] = top == -INFINITY ? 0.0f : top;
                                l[nt][e] *= f[e];
                                if (!each) {
                                    f[e] *= ratio;
                                    continue;
                                }
                                float big = fmaxf(s[nt][e] == -INFINITY ? 0.0f : sv0, s[nt][e + 2] == -INFINITY ? 0.0f : sv1);
#pragma unroll
                                for (int d = 4; d < 32; d *= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
                                float *own = &row_unit[warp][8 * nt + 2 * j + e];
                                const float old = apart ? *own : before, now = fmaxf(old, pow2_above(big));
                                f[e] *= old * pow2_inverse(now);
                                __syncwarp();
                                if (g == 0) *own = now;
                            }
#pragma unroll
                            for (int st = 0; st < S::kSteps; ++st)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[nt][st][e] *= f[e & 1];
                        }
                        if (each) absent |= kApart;
                        __syncwarp();
                    }
                    w0 *= (float)(1 << kAttnRoom), w1 *= (float)(1 << kAttnRoom);
                    uint32_t p[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float p0 = ex2(s[nt][0] - ref[nt][0]), p1 = ex2(s[nt][1] - ref[nt][1]);
                        const float p2 = ex2(s[nt][2] - ref[nt][0]), p3 = ex2(s[nt][3] - ref[nt][1]);
                        l[nt][0] += p0 + p2, l[nt][1] += p1 + p3;
                        float y[4] = {p0 * w0, p1 * w0, p2 * w1, p3 * w1};
                        if (!whole && (absent & kApart)) {  // hidden: the scale over the row's unit may be more than fp32 holds
                            const float z[4] = {p0, p1, p2, p3};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float per = pow2_inverse(row_unit[warp][8 * nt + 2 * j + (e & 1)]);
                                const float w = (e < 2 ? sv0 : sv1) * per * (float)(1 << kAttnRoom);
                                y[e] = s[nt][e] == -INFINITY ? 0.0f : z[e] * w;
                            }
                        }
                        const __half2 lo = __floats2half2_rn(y[0], y[1]), hi = __floats2half2_rn(y[2], y[3]);
                        p[nt][0] = transposed(*reinterpret_cast<const uint32_t *>(&lo));
                        p[nt][1] = transposed(*reinterpret_cast<const uint32_t *>(&hi));
                    }
                    // V of tokens 2j, 2j + 1, 2j + 8, 2j + 9, the lane's channels
                    uint32_t vw[4][S::kVWords];
                    constexpr int step_v = S::kVWords < 4 ? S::kVWords : 4;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int w = 0; w < S::kVWords; w += step_v)
                            lds<step_v>(k_at + v_off[e & 1][w / 4] + (e >> 1) * eight, vw[e] + w);
                    [[maybe_unused]] Zero za, zb;
                    if constexpr (U4) {
                        const uint2 ta = lds64(w_at + 64 + 8 * j), tb = lds64(w_at + 64 + 8 * j + 32);
                        za = zero_of(ta.x & 15u, ta.y & 15u);
                        zb = zero_of(tb.x & 15u, tb.y & 15u);
                    }
#pragma unroll
                    for (int w = 0; w < S::kVWords; ++w) {
                        if constexpr (U4) {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint32_t ra[4], rb[4];
                                u4_pairs(prmt(vw[0][w], vw[1][w], half ? 0x7632 : 0x5410), za, ra);
                                u4_pairs(prmt(vw[2][w], vw[3][w], half ? 0x7632 : 0x5410), zb, rb);
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const uint32_t f[4] = {ra[2 * e], ra[2 * e + 1], rb[2 * e], rb[2 * e + 1]};
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][4 * w + 2 * half + e], f, p[nt][0], p[nt][1]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                // the tokens' codes of a channel side by side: a0 b0 a1 b1
                                const uint32_t ta = prmt(vw[0][w], vw[1][w], half ? 0x7362 : 0x5140);
                                const uint32_t tb = prmt(vw[2][w], vw[3][w], half ? 0x7362 : 0x5140);
                                uint32_t f[4];
                                s8_pairs(ta, f[0], f[1]);
                                s8_pairs(tb, f[2], f[3]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][2 * w + half], f, p[nt][0], p[nt][1]);
                            }
                        }
                    }
                }
                __syncwarp();  // the stage has been read
                ask(stage);
                if (++stage == ST) stage = 0;
                if constexpr (!whole) pos0 += kAttnChunk;
            }
        };
        const int units = (int)(end - x), room = seen_by_all - 16 - pos0;
        const int all = room < 0 ? 0 : min(units, room / kAttnChunk + 1);
        tiles(std::true_type{}, all);
        pos0 += all * kAttnChunk;
        if (units > all) tiles(std::false_type{}, units - all);
        x = end;
        at.chunk = at.units - 1;  // (where this is not so, nothing follows)
        if (x < share.to) next(a, at, S::kRows);
        // the warps' parts meet
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                const int r = 8 * nt + 2 * j + e;
                const float unit = absent & kApart ? row_unit[warp][r] : pow2_inverse(per_unit);
                if (g == 0) stats[warp][r] = make_float4(m[nt][e], unit, l[nt][e], 0.0f);
            }
        __syncthreads();
        const bool done = starts_here && ends_here;
        float *slot = attn_slot(a, blockIdx.x, starts_here ? 1 : 0, S::kRows, DP);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + 2 * j + e;
                float top = -INFINITY, top_unit = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 o = *reinterpret_cast<const float2 *>(&stats[w][r]);
                    top = fmaxf(top, o.x), top_unit = fmaxf(top_unit, o.y);
                }
                const float shrink = stats[warp][r].y * pow2_inverse(top_unit);
                const float f = (m[nt][e] == top ? 1.0f : ex2(m[nt][e] - top)) * shrink;
                float *to = join + (warp * 8 + 2 * j + e) * S::kPitch + g;
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
                    for (int half = 0; half < 2; ++half) to[(2 * s + half) * 8] = acc[nt][s][2 * half + e] * f;
            }
            __syncthreads();
            // pairs of channels of a row, in the order of (step, half, g)
            for (int i = threadIdx.x; i < 8 * DP / 2; i += kThreads) {
                const int r = i / (DP / 2), p = i % (DP / 2), row = 8 * nt + r;
                if (row >= width) break;
                const int step = p / 8, pg = p % 8;
                float v0 = 0.0f, v1 = 0.0f, top = -INFINITY, total = 0.0f, top_unit = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float *from = join + (w * 8 + r) * S::kPitch + 16 * step + pg;
                    v0 += from[0], v1 += from[8];
                    const float2 o = *reinterpret_cast<const float2 *>(&stats[w][row]);
                    top = fmaxf(top, o.x), top_unit = fmaxf(top_unit, o.y);
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 o = stats[w][row];
                    total += o.z * (o.x == top ? 1.0f : ex2(o.x - top));
                }
                const int d = sum_channel<U4, DP>(pg, step, 0);
                if (!done) {
                    *reinterpret_cast<float2 *>(slot + row * DP + d) = make_float2(v0, v1);
                    if (p == 0) {
                        slot[S::kRows * DP + 2 * row] = top, slot[S::kRows * DP + 2 * row + 1] = total;
                        slot[S::kRows * (DP + 2) + row] = top_unit;
                    }
                } else if (d < c.D) {
                    attn_store(a, first, head, row0 + row, d, v0, v1, top, total, top_unit * kAttnWeightUnit);
                }
            }
            __syncthreads();
        }
    }
}

template <bool U4, int DP, int NT>
qnn_status launch(KvAttnArgs a, cudaStream_t s)
{
    using S = Shape<U4, DP, NT>;
    auto kern = kv_attn_few_kernel<U4, DP, NT>;
    static std::atomic<uint64_t> opted_in{0};
    // of an SM's 228 KB: 1 KB a block for the system, and the static part
    constexpr int kMost = (S::kMinBlocks == 2 ? 112 : 224) << 10, kStatic = 12 << 10;
    const int join = kWarps * 8 * S::kPitch * 4, sums = (a.c.batch + 1) * 8 + 128, stage = kWarps * stage_bytes(a.c.row_bytes);
    a.stages = std::min(8, (kMost - kStatic - join - sums) / stage);
    if (!opt_in_smem(kern, kMost - kStatic, opted_in, 100)) return QNN_ERR_CUDA;
    return kv_launch(kern, dim3((unsigned)a.blocks), kThreads, join + sums + a.stages * stage, s, a);
}

template <bool U4>
qnn_status launch_channels(const KvAttnArgs &a, const AttnPlan &p, cudaStream_t s)
{
    if (p.channels == 64) return p.rows == 8 ? launch<U4, 64, 1>(a, s) : launch<U4, 64, 2>(a, s);
    if (p.channels == 128) return launch<U4, 128, 1>(a, s);
    return p.rows == 8 ? launch<U4, 256, 1>(a, s) : launch<U4, 256, 2>(a, s);
}

}  // namespace

AttnPlan attn_few_plan(const KvArgs &c, int group)
{
    AttnPlan p;
    p.channels = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
    const int64_t rows = (int64_t)c.tokens * group;
    p.rows = rows <= 8 ? 8 : 16;  // with 128 channels: 8 at most come here
    p.blocks = std::min(kAttnMaxBlocks, sm_count() * (p.rows * p.channels <= 1024 ? 2 : 1));
    return p;
}

qnn_status launch_attn_few(const KvAttnArgs &a, const AttnPlan &p, bool u4, cudaStream_t s)
{
    return u4 ? launch_channels<true>(a, p, s) : launch_channels<false>(a, p, s);
}

}  // namespace qnn
