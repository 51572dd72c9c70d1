// qnn_kv_attn.cuh -- what the kernels of q_kv_attn share: the arguments, how the work is
// divided, and the workspace in which parts of a row's sum meet.
#pragma once
#include "qnn_kv.cuh"

namespace qnn {

struct KvAttnArgs {
    KvArgs c;
    const void *q;
    void *out;
    float *lse;
    const uint32_t *mask;
    float *ws;
    int64_t ld_q, ld_out;
    float scale_log2;  // scale * log2(e)
    int heads_q, group, mask_words, bf16;
    int t_min, t_max;  // sequences with fewer or more newest tokens are not this launch's
    int blocks;        // of the attention's grid
    int stages;        // of a ring
};

// The work: an item is a sequence's tile of rows (rows t * group + g, t a newest token, g one of
// the heads of q that share a head of the cache) with one head of the cache; its units are chunks
// of 128 tokens, as far as the tile sees.  All units stand in one line, by sequence, row tile,
// head and position, and each block has an equal part of it, whatever the lengths: an item that
// lies in one block is finished there; one that goes on behind a block's end is finished by the
// joining kernel, from one part of each block.
//
// Workspace: for each block a record of 8 ints (of the item that begins in its part of the line and
// goes on behind it: attn_record), then two
// slots of parts: slot 0 for an item that began in an earlier block, slot 1 for one that begins
// here and goes on.  A slot: [rows][channels] sums, then for each row the maximum and the sum of
// weights, then for each row the unit of V's scales.
constexpr int kAttnRecord = 8, kAttnChunk = 128;

// Weights are p * (scale of V / unit) * 2^kAttnRoom in f16: p <= 2^kAttnSlack, as maxima move only when a
// score passes them by more, and scale <= unit, so that they stay below 2^16; a row's unit is a power
// of two no smaller than any scale that the row has seen so far: the tokens that are hidden from it have no
// part in it.  Rows differ in what they see only at the end of an item, and their units are one until a token there
// that some rows do not see has a scale above it; then each has its own.
constexpr int kAttnSlack = 8, kAttnRoom = 7;
constexpr float kAttnWeightUnit = 1.0f / (1 << kAttnRoom);

__host__ __device__ inline int64_t attn_slot_floats(int rows, int channels) { return (int64_t)rows * (channels + 3); }

__device__ __forceinline__ float *attn_slot(const KvAttnArgs &a, int block, int slot, int rows, int channels)
{
    return a.ws + (int64_t)a.blocks * kAttnRecord + (2 * (int64_t)block + slot) * attn_slot_floats(rows, channels);
}

// The block's record: `last` is the block in which the item ends, < 0 where no item begins here and
// goes on.  The item's rows are rows row0 .. row0 + width - 1 of those of its sequence.
__device__ __forceinline__ void attn_record(const KvAttnArgs &a, int last, int64_t first, int row0, int width, int head)
{
    int4 *record = reinterpret_cast<int4 *>(a.ws) + 2 * blockIdx.x;
    record[0] = make_int4(last, head, row0, width);
    *reinterpret_cast<int64_t *>(record + 1) = first;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
    return d;
}

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// f16 magic numbers: 0x6400 | u is 1024 + u; for the upper half of a byte 1024 + 16 u, of which
// a sixteenth is 64 + u.
constexpr uint32_t kMagic = 0x64006400u, kOne = 0x3c003c00u, kSixteenth = 0x2c002c00u;
constexpr uint32_t k1152 = 0x64806480u;

// Four s8 codes (as q + 128) of a row to two registers of neighbouring pairs.
__device__ __forceinline__ void s8_pairs(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    lo = hsub2_u32(prmt(w, kMagic, 0x7150), k1152);
    hi = hsub2_u32(prmt(w, kMagic, 0x7352), k1152);
}

struct Zero {
    uint32_t lo, hi;  // -(1024 + z), -(64 + z)
};

__device__ __forceinline__ Zero zero_of(uint32_t z0, uint32_t z1)
{
    const uint32_t z = z0 | z1 << 16;
    return {0xe400e400u + z, 0xd400d400u + (z << 4)};
}

// The halves' four 4-bit codes each, less their zero points, as four registers.
__device__ __forceinline__ void u4_pairs(uint32_t w, const Zero &z, uint32_t (&r)[4])
{
    const uint32_t v = w >> 8;
    r[0] = fma2(and_or(w, 0x000f000fu, kMagic), kOne, z.lo);
    r[1] = fma2(and_or(w, 0x00f000f0u, kMagic), kSixteenth, z.hi);
    r[2] = fma2(and_or(v, 0x000f000fu, kMagic), kOne, z.lo);
    r[3] = fma2(and_or(v, 0x00f000f0u, kMagic), kSixteenth, z.hi);
}

// 2^k as fp32, -126 <= k <= 127
__device__ __forceinline__ float pow2i(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// Of a power of two from 2^-126 to 2^126, its inverse; the power of two that is no smaller than v, and 2^126 at most.
__device__ __forceinline__ float pow2_inverse(float v) { return __uint_as_float(0x7f000000u - __float_as_uint(v)); }
__device__ __forceinline__ float pow2_above(float v) { return __uint_as_float((__float_as_uint(v) + 0x7fffffu) & 0xff800000u); }

// A row of q is brought near f16's largest by a power of two, 2^-113 .. 2^141 for 16-bit types, in two exact
// steps; its inverse multiplies K's scales (which have the call's scale in them), a subnormal at the least, and
// their product the sums: so nothing on the way is far from the scores or from what K's scales are.
struct RowUnit {
    float up0, up1, down;
    __device__ __forceinline__ explicit RowUnit(float top)  // the row's largest
    {
        const int e2 = (int)(__float_as_uint(top) >> 23), k = top == 0.0f || e2 == 255 ? 0 : 14 + 127 - e2;
        up0 = pow2i(k >> 1), up1 = pow2i(k - (k >> 1));
        down = pow2i(-(k >> 1)) * pow2i((k >> 1) - k);
    }
    __device__ __forceinline__ float up(float v) const { return v * up0 * up1; }
};

// The units that a tile of `width` rows, number rt, sees of a sequence; one at least, so that
// rows that see nothing are written too.
__device__ __forceinline__ int attn_units(const KvAttnArgs &a, int T, int len, int rt, int width)
{
    int seen = len;
    if (!a.mask) {
        const int last = min((rt + 1) * width, T * a.group) - 1;  // all rows of a call are fewer than 2^31
        seen = len - T + last / a.group + 1;
    }
    return max(1, (seen + kAttnChunk - 1) / kAttnChunk);
}

__device__ __forceinline__ int attn_row_tiles(const KvAttnArgs &a, int T, int width)
{
    return (T * a.group + width - 1) / width;
}

// Sequence b, without newest tokens where they are not this launch's.
__device__ __forceinline__ KvSeq attn_seq(const KvAttnArgs &a, int b)
{
    KvSeq s = kv_seq(a.c, b);
    if (s.T < a.t_min || s.T > a.t_max) s.T = 0;
    return s;
}

// A sequence's units.
__device__ __forceinline__ int64_t attn_weight(const KvAttnArgs &a, const KvSeq &s, int width)
{
    if (s.T <= 0) return 0;
    const int tiles = attn_row_tiles(a, s.T, width);
    int64_t n = 0;
    if (a.mask || tiles == 1) n = (int64_t)tiles * attn_units(a, s.T, s.len, tiles - 1, width);
    else
        for (int rt = 0; rt < tiles; ++rt) n += attn_units(a, s.T, s.len, rt, width);
    return n * a.c.heads;
}

// Where a unit stands.
struct AttnCursor {
    int64_t first;
    int b, rt, h, chunk, units, tiles, T, len;
};

__device__ __forceinline__ void attn_sequence(const KvAttnArgs &a, AttnCursor &c, int width)
{
    const KvSeq s = attn_seq(a, c.b);
    c.T = s.T;
    c.len = s.len;
    c.first = s.first;
    c.tiles = attn_row_tiles(a, c.T, width);
}

// The cursor at unit x of the line, whose sums up to each sequence are `sums`.
__device__ __forceinline__ AttnCursor attn_find(const KvAttnArgs &a, const int64_t *sums, int64_t x, int width)
{
    AttnCursor c;
    int lo = 0, hi = a.c.batch - 1;  // the last sequence that begins at or before x
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (sums[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    c.b = lo;
    attn_sequence(a, c, width);
    x -= sums[lo];
#pragma unroll 1
    for (c.rt = 0;; ++c.rt) {
        c.units = attn_units(a, c.T, c.len, c.rt, width);
        const int64_t n = (int64_t)c.units * a.c.heads;
        if (x < n || c.rt + 1 >= c.tiles) break;
        x -= n;
    }
    c.h = (int)(x / c.units);
    c.chunk = (int)(x - (int64_t)c.h * c.units);
    return c;
}

// The cursor at the first unit of the next row tile.
__device__ __forceinline__ AttnCursor attn_next_rows(const KvAttnArgs &a, AttnCursor c, int width)
{
    c.h = 0;
    if (++c.rt >= c.tiles) {
        c.rt = 0;
#pragma unroll 1
        do {
            if (++c.b >= a.c.batch) return c;
            attn_sequence(a, c, width);
        } while (c.T <= 0);
    }
    c.units = attn_units(a, c.T, c.len, c.rt, width);
    return c;
}

__device__ __forceinline__ void attn_next(const KvAttnArgs &a, AttnCursor &c, int width)
{
    if (++c.chunk < c.units) return;
    c.chunk = 0;
    if (++c.h >= a.c.heads) c = attn_next_rows(a, c, width);
}

// sums[i]: the units of sequences 0 .. i - 1, by all threads of a block; returns all of them.
template <int THREADS>
__device__ __forceinline__ int64_t attn_sums(const KvAttnArgs &a, int64_t *sums, int width)
{
    __shared__ int64_t part[THREADS / 32];
    const int per = (a.c.batch + THREADS - 1) / THREADS, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b0 = min((int)threadIdx.x * per, a.c.batch), b1 = min(b0 + per, a.c.batch);
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t w = attn_weight(a, attn_seq(a, b), width);
        sums[b] = own;
        own += w;
    }
    int64_t upto = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) part[warp] = upto;
    __syncthreads();
    int64_t before = upto - own, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += part[w];
        all += part[w];
    }
    for (int b = b0; b < b1; ++b) sums[b] += before;
    if (threadIdx.x == 0) sums[a.c.batch] = all;
    __syncthreads();
    return all;
}

// A block's part of the line: [from, to), of `all` units over `active` blocks.
struct AttnShare {
    int64_t all, from, to;
    int active;
    __device__ __forceinline__ AttnShare(int64_t n, int blocks, int block) : all(n)
    {
        active = (int)min((int64_t)blocks, n);
        from = block < active ? n * block / active : n;
        to = block < active ? n * (block + 1) / active : n;
    }
    __device__ __forceinline__ int block_of(int64_t x) const { return (int)(((x + 1) * active - 1) / all); }
};

// 16 bytes global -> shared, asynchronously.  Whole warps copy this way: bulk copies of lanes that each
// have an address of their own are issued one lane after the other, 20 instructions each.
__device__ __forceinline__ void copy_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the thread's last n groups of copies have landed.
__device__ __forceinline__ void copies_wait(int n)
{
    switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
    }
}

// The page of 16-token tile `tile` of sequence b, or -1.
__device__ __forceinline__ int attn_page(const KvAttnArgs &a, int b, int tile, int *in_page)
{
    return kv_page(a.c, b, kv_page_index(a.c, tile, in_page));
}

// Whether newest token t's row sees position p.
__device__ __forceinline__ bool attn_sees(const KvAttnArgs &a, const AttnCursor &c, int t, int p)
{
    if (p >= c.len) return false;
    const int j = p - (c.len - c.T);
    if (j < 0) return true;
    if (!a.mask) return j <= t;
    if ((j >> 5) >= a.mask_words) return false;
    return (a.mask[(c.first + t) * a.mask_words + (j >> 5)] >> (j & 31)) & 1u;
}

__device__ __forceinline__ uint32_t attn_pack(const KvAttnArgs &a, float x, float y)
{
    if (a.bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float attn_lse(float m, float total)
{
    return total == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(m, log2f(total)), 0.6931471805599453f);
}

// Row r of an item (of a sequence whose newest tokens begin at row `first`), channels d and d + 1
// of it, from sums of weights and codes in units of `unit`; with d = 0, its logarithm.
__device__ __forceinline__ void attn_store(const KvAttnArgs &a, int64_t first, int head, int r, int d, float v0, float v1,
                                           float m, float total, float unit)
{
    const int t = r / a.group;
    const int64_t row = first + t;
    const int hq = head * a.group + (r - t * a.group);
    const float o0 = total == 0.0f ? 0.0f : v0 / total * unit, o1 = total == 0.0f ? 0.0f : v1 / total * unit;
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + row * a.ld_out + (int64_t)hq * a.c.D + d) =
        attn_pack(a, o0, o1);
    if (d == 0 && a.lse) a.lse[row * a.heads_q + hq] = attn_lse(m, total);
}

// The row tile, channels and blocks of a call's kernel.
constexpr int kAttnMaxBlocks = 320;
struct AttnPlan {
    int rows, channels, blocks;
};

AttnPlan attn_few_plan(const KvArgs &c, int group);
AttnPlan attn_rows_plan(const KvArgs &c, int group);
qnn_status launch_attn_rows(const KvAttnArgs &a, const AttnPlan &p, bool u4, cudaStream_t s);
qnn_status launch_attn_few(const KvAttnArgs &a, const AttnPlan &p, bool u4, cudaStream_t s);

}  // namespace qnn
