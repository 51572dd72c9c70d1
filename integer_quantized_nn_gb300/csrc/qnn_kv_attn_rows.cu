// qnn_kv_attn_rows.cu -- q_kv_attn for many rows of a head of the cache: trees of drafted tokens
// and chunks of prompts, 128 rows (the heads of q that share a head of the cache, times newest
// tokens) at a time on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = e^(S - m),  O += P V
// for chunks of 128 tokens.  There are two streams with a maximum, a sum and an O of their own (S and O of both
// fill tensor memory): two tiles of rows over the same chunks, or the even and odd chunks of one tile,
// which meet where an item ends.  The rows' warps have the streams in turn: while they make P of one, the
// tensor cores work on the other's.
//
// A chunk of 2048 tokens over 8192, 32 heads on 8, D = 128, in 8 bits takes 279 us, 862 TFLOP/s (45% of the
// library's bf16 products); 8 trees of 64 tokens over 8192 take 106 us; with D = 256, 16 heads on 8, the chunk
// takes 320 us, 751 TFLOP/s (a tile of K or V is then made while nothing multiplies by it).  Of the 2800 cycles
// of a step (D = 128) the rows' warps work in 1850, the tensor cores in 1200; an item's start and end (q to f16, the
// sums out) take 6 us in which the tensor cores wait.
//
// Roles of a block's warps:
//   0       places: which pages hold a chunk of 128 tokens, and which item comes next
//   1       MMA: S of a chunk, then O of the same stream's chunk before ... in order
//   2, 3    scales: of K for the scores; of V over a unit for the weights
//   4..7    codes: global -> registers -> f16 integers -> the swizzled operand tiles, for K (K-major)
//           and V (N-major) the same image
//   8..15   rows: 16 rows of S each, in tensor memory -> weights as f16 over it; the other way for O
//           when a maximum has moved by more than 2^8 or the unit has grown
#include "qnn_kv_attn.cuh"

namespace qnn {
namespace {

constexpr int kRows = 128, kTokens = kAttnChunk, kThreads = 512, kInfos = 4;
constexpr int kCodeWarp0 = 4, kCodeWarps = 4, kRowWarp0 = 8, kRowWarps = 8;
constexpr uint32_t kTmemCols = 512, kOCol = 256;  // S of both streams, then O

// An item, or the part of one that is this block's, as the copies' warp leaves it to the others.
struct Item {
    int64_t first;              // row of the sequence's first newest token
    int b, rt, h, chunk;        // chunk: the first
    int count, units, T, len;   // count: of chunks here; units: of the item
};
constexpr int kItems = 4;

// Where 16 tokens of a chunk are: bytes from the first page to their K rows and their K words; words -1:
// they are not there, and rows are those of some place in the cache.
struct Tile16 {
    int64_t rows, words;
};
constexpr int kPlaces = 8;

// Of a chunk: scales of K times the call's, and of V over the stream's unit, for two tokens together (k k v v).
// kWhole: all rows see all of it.  kApart: some rows do not see a token whose scale is above the unit; V's scales
// are as in the cache, and each row has a unit of its own from there to the item's end.
struct Info {
    float scales[kTokens / 2][4];
    float ratio, unit, before;  // the unit before over this one; this one; the one before
    uint32_t present;           // 16-token tiles that are there, in bits 0..7
};
constexpr uint32_t kWhole = 0x1ffu, kApart = 0x200u;

// f16 operands, A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Tensor memory as fragments: 16 lanes; registers 4 i .. 4 i + 3 of thread 4 g + j are row g, columns
// 8 i + 2 j and + 1, then the same of row g + 8 (16x256b); register 2 i + h is row g + 8 h, column
// 4 i + j (16x128b): two f16 of the first are one word of the second.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 "
        "[%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x16.b32 "
        "[%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// a lane's row, 8 columns
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// The tile image as an operand whose rows are K: 64 of N (128 bytes) a row, 8 rows an atom of the
// 128-byte swizzle; the next 8 rows follow, the next 64 of N are `panel` bytes on.
__device__ __forceinline__ uint64_t sdesc_n_major(uint32_t addr, uint32_t panel)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((panel >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// 16 bytes of shared memory that nothing writes meanwhile: the compiler may read them early
__device__ __forceinline__ uint4 lds_scales(uint32_t at)
{
    uint4 v;
    asm("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

// the lowest n bits, n from 0 (or below) to 32 (or above)
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }

// Which of positions p0 .. p0 + 31 the row of newest token t sees.
__device__ __forceinline__ uint32_t seen_bits(const KvAttnArgs &a, const Item &c, int t, int p0)
{
    const int base = c.len - c.T;
    if (!a.mask) return low_bits(min(c.len, base + t + 1) - p0);
    const int j0 = p0 - base, w = j0 >> 5;
    const uint32_t *m = a.mask + (c.first + t) * a.mask_words;
    const uint32_t lo = w >= 0 && w < a.mask_words ? m[w] : 0u, hi = w + 1 >= 0 && w + 1 < a.mask_words ? m[w + 1] : 0u;
    return (low_bits(-j0) | __funnelshift_r(lo, hi, j0 & 31)) & low_bits(c.len - p0);
}

// A warp's 16 rows of S of a chunk -> P over it.  A thread has 2 rows (8 q + g) and the columns 8 i + 2 j and + 1 of
// each: with a row to a thread each would read all scales of the chunk from shared memory, 1500 cycles
// of its bandwidth a chunk.  scales: of K and V, of the thread's first two columns; bits: lanes t and t + 16 have
// those of the positions that row t sees; unit: of each row, APART; sums_still: waits until no product adds to the sums.
template <bool MASKED, bool APART, int DP, typename F>
__device__ __forceinline__ void weights(uint32_t s_at, uint32_t o_at, uint32_t scales, const uint32_t (&bits)[4], int j,
                                        bool first, float ratio, const float (&cr)[2], float (&m)[2], float (&l)[2],
                                        float *unit, const F &sums_still)
{
    const int g = (threadIdx.x & 31) >> 2;
    uint32_t b[2][4], p[32];
    if constexpr (MASKED) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int w = 0; w < 4; ++w) b[q][w] = __shfl_sync(0xffffffffu, bits[w], 8 * q + g) >> (2 * j);
    }
    // The maxima so far are tried first: a thread's 32 weights of a row whose sum stays below 2^8 are
    // all below it.  New maxima are looked for where they do not, at first and with a new unit.  A row that has
    // seen nothing yet has the maximum -inf: its weights are infinite, so that they do not, or hidden.
    bool fresh = MASKED || first || ratio != 1.0f;
    float2 s[2];
#pragma unroll 1
    for (;;) {
        uint32_t v[64];
        if (fresh) {
            float top[2] = {-INFINITY, -INFINITY}, f[2], big[2] = {0.0f, 0.0f};
            tmem_ld_frag(s_at, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint4 kw = lds_v4(scales + 64 * i);
                const float2 k = as_f2(kw.x, kw.y);
                const uint32_t bit = 1u << (8 * (i & 3));
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float2 y = mul2(as_f2(v[4 * i + 2 * q], v[4 * i + 2 * q + 1]), mul2(k, both(cr[q])));
                    if constexpr (MASKED) {
                        y.x = b[q][i >> 2] & bit ? y.x : -INFINITY;
                        y.y = b[q][i >> 2] & (2 * bit) ? y.y : -INFINITY;
                    }
                    if constexpr (APART)
                        big[q] = max3(big[q], b[q][i >> 2] & bit ? __uint_as_float(kw.z) : 0.0f,
                                      b[q][i >> 2] & (2 * bit) ? __uint_as_float(kw.w) : 0.0f);
                    top[q] = max3(top[q], y.x, y.y);
                }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                top[q] = fmaxf(top[q], __shfl_xor_sync(0xffffffffu, top[q], 1));
                top[q] = fmaxf(top[q], __shfl_xor_sync(0xffffffffu, top[q], 2));
                const float u = fmaxf(m[q], top[q]);
                f[q] = m[q] == -INFINITY ? 0.0f : ex2(m[q] - u);
                m[q] = u;
                l[q] *= f[q];
                if constexpr (APART) {
                    big[q] = fmaxf(big[q], __shfl_xor_sync(0xffffffffu, big[q], 1));
                    big[q] = fmaxf(big[q], __shfl_xor_sync(0xffffffffu, big[q], 2));
                    const float now = fmaxf(unit[q], pow2_above(big[q]));
                    f[q] *= unit[q] * pow2_inverse(now);
                    unit[q] = now;
                } else {
                    f[q] *= ratio;
                }
            }
            if (!first && __any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
                sums_still();
#pragma unroll 1
                for (int at = 0; at < DP; at += 32) {
                    uint32_t o[16];
                    tmem_ld_frag(o_at + at, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (e & 2 ? f[1] : f[0]));
                    tmem_st_frag(o_at + at, o);
                }
            }
        }
        tmem_ld_frag(s_at, v);
        tmem_ld_wait();
        s[0] = s[1] = both(0.0f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint4 kw = lds_scales(scales + 64 * i);
            const float2 k = as_f2(kw.x, kw.y), w = as_f2(kw.z, kw.w);
            const uint32_t bit = 1u << (8 * (i & 3));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float2 y = fma2(as_f2(v[4 * i + 2 * q], v[4 * i + 2 * q + 1]), mul2(k, both(cr[q])), both(-m[q]));
                y.x = ex2(y.x), y.y = ex2(y.y);
                if constexpr (MASKED) {
                    y.x = b[q][i >> 2] & bit ? y.x : 0.0f;
                    y.y = b[q][i >> 2] & (2 * bit) ? y.y : 0.0f;
                }
                s[q] = add2(s[q], y);
                if constexpr (APART) {  // hidden: the scale over the row's unit may be more than fp32 holds
                    float2 v = mul2(w, both(pow2_inverse(unit[q])));
                    v.x = b[q][i >> 2] & bit ? v.x : 0.0f;
                    v.y = b[q][i >> 2] & (2 * bit) ? v.y : 0.0f;
                    y = mul2(mul2(y, both((float)(1 << kAttnRoom))), v);
                } else {
                    y = mul2(y, w);
                }
                const __half2 h = __floats2half2_rn(y.x, y.y);
                p[2 * i + q] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        s[0].x += s[0].y, s[1].x += s[1].y;
        if (fresh) break;
        fresh = __any_sync(0xffffffffu, s[0].x > (float)(1 << kAttnSlack) || s[1].x > (float)(1 << kAttnSlack));
        if (!fresh) break;
    }
    tmem_st_pairs(s_at, p);
    l[0] += s[0].x, l[1] += s[1].x;
}

// PAIR: the streams are two tiles of rows over the same chunks, which are converted once for both.
// Of more than 128 channels (never PAIR) tensor memory has room for one O and shared memory for one tile of K and
// one of V: even and odd chunks have an S each, and one maximum, sum and O.
template <bool U4, int DP, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_rows_kernel(const __grid_constant__ KvAttnArgs a)
{
    constexpr uint32_t PANEL = kTokens * 128, TILE = PANEL * (DP / 64);
    constexpr int ROWS = PAIR ? 2 * kRows : kRows;  // of an item
    constexpr bool ONE = DP > 128, SPLIT = !PAIR && !ONE;  // SPLIT: the streams' parts of a row meet at the end
    constexpr int TILES = ONE ? 1 : 2;                      // of K, and of V
    const KvArgs &c = a.c;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ __align__(8) uint64_t place_full[kPlaces], place_empty[kPlaces], tile_full[4], tile_empty[4],
        info_full[kInfos], info_empty[kInfos], item_full[kItems], item_empty[kItems], s_full[2], p_ready[2], q_full, o_full,
        o_added, mma_end;
    __shared__ __align__(16) Info infos[kInfos];
    __shared__ __align__(16) Tile16 places[kPlaces][kTokens / 16];
    __shared__ Item items[kItems];
    __shared__ float row_m[2][kRows], row_l[2][kRows], row_top[2][kRows], row_c[2][kRows], row_unit[2][kRows];
    __shared__ uint32_t present[kPlaces], tmem_slot;  // 16-token tiles of a chunk that are there
    uint8_t *smem = raw + (-smem_u32(raw) & 1023u);  // the swizzle's atoms
    // tiles: K of even and odd chunks, V of both (ONE: of any); q (of both streams); the sums of the line
    const uint32_t tiles = smem_u32(smem), q_tile = tiles + 2 * TILES * TILE;
    int64_t *sums = reinterpret_cast<int64_t *>(smem + (2 * TILES + (PAIR ? 2 : 1)) * TILE);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPlaces; ++i) {
            mbar_init(smem_u32(&place_full[i]), 1);
            mbar_init(smem_u32(&place_empty[i]), kCodeWarps + 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&tile_full[i]), kCodeWarps / 2);
            mbar_init(smem_u32(&tile_empty[i]), 1);
        }
        for (int i = 0; i < kInfos; ++i) {
            mbar_init(smem_u32(&info_full[i]), 2);
            mbar_init(smem_u32(&info_empty[i]), kRowWarps);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(smem_u32(&item_full[i]), 1);
            mbar_init(smem_u32(&item_empty[i]), kRowWarps + 3);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_ready[i]), kRowWarps);
        }
        mbar_init(smem_u32(&q_full), kRowWarps);
        mbar_init(smem_u32(&o_full), 1);
        mbar_init(smem_u32(&o_added), 1);
        mbar_init(smem_u32(&mma_end), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // only now: a block of the next grid that took tensor memory first and waited for this grid
    // would keep it from blocks of this one
    grid_dependency_launch();
    grid_dependency_wait();

    // Nothing for the join until an item's parts are stored: it trusts the record, and a block whose waits gave up
    // must not leave it what an earlier call, or nobody, wrote there.  (attn_sums has a barrier behind this.)
    if (threadIdx.x == 0) attn_record(a, -1, 0, 0, 0, 0);
    const AttnShare share(attn_sums<kThreads>(a, sums, ROWS), a.blocks, blockIdx.x);
    const int chunks = (int)(share.to - share.from);

    bool ok = true;
    auto release = [&](uint64_t &bar) {  // what the warp has read may be written again
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar));
    };
    auto wait = [&](uint64_t &bar, int use) {  // the use-th phase of a barrier, by a whole warp
        ok = ok && __all_sync(0xffffffffu, mbar_wait_short(smem_u32(&bar), (uint32_t)use & 1u, nullptr));
        return ok;  // a wait that gave up is reported at the end
    };

    // Registers so that no loop spills: the tiles leave the L1 a few KB, and a spilled word comes from the L2 (the
    // prompt of the note above: 296 us, and 316 with 56, 104 and 176).
    // 128 registers a thread at the launch, and as many after: 80 + 128 + 2 * 152 = 4 * 128
    if (warp < kCodeWarp0) {
    regs_dec<80>();
    if (chunks <= 0) {
    } else if (warp == 0) {
        AttnCursor at = attn_find(a, sums, share.from, ROWS);
        int left = 0, item = 0;
#pragma unroll 1
        for (int n = 0; n < chunks && ok; ++n) {
            if (left == 0) {
                const int slot = (unsigned)item % kItems;
                if (item >= kItems && !wait(item_empty[slot], (unsigned)item / kItems - 1)) break;
                left = min(at.units - at.chunk, chunks - n);
                if (lane == 0) {
                    items[slot] = {at.first, at.b, at.rt, at.h, at.chunk, left, at.units, at.T, at.len};
                    mbar_arrive(smem_u32(&item_full[slot]));
                }
                ++item;
            }
            --left;
            const int slot = (unsigned)n % kPlaces, tile = at.chunk * (kTokens / 16) + lane;
            Tile16 place = {0, -1};
            if (lane < kTokens / 16 && tile * 16 < at.len) {
                int in_page;
                const int page = attn_page(a, at.b, tile, &in_page);
                if (page >= 0) {
                    const int64_t head = page * c.page_bytes + (int64_t)at.h * c.head_bytes;
                    place = {head + in_page * 16 * c.row_bytes, head + 2 * c.page * c.row_bytes + in_page * 64};
                }
            }
            if (n >= kPlaces && !wait(place_empty[slot], (unsigned)n / kPlaces - 1)) break;
            const uint32_t there = __ballot_sync(0xffffffffu, place.words >= 0);
            if (lane < kTokens / 16) places[slot][lane] = place;
            if (lane == 0) present[slot] = there;
            release(place_full[slot]);
            if (n + 1 < chunks) attn_next(a, at, ROWS);
        }
    } else if (warp == 1) {
        const uint32_t idesc_s = idesc_f32acc(0, 0, kRows, kTokens);
        const uint32_t idesc_o = idesc_f32acc(0, 0, kRows, 0) | (uint32_t)(c.D >> 3) << 17 | 1u << 16;  // B is N-major
        // Step by step: S of step t after O of step t - 2, which is of the same stream.  One lane issues products and
        // commits, always the same, but all lanes go through the loops: a product's descriptors are one value for the
        // warp, and so no lane has another, however the compiler lays out the branches.  (Where one lane went through
        // the loops alone, an unrolled loop with a condition inside read operands elsewhere.  With the lane chosen by
        // its number, which does not tell the compiler that it is one, the prompt of the note above took 327 us.)
        const uint64_t kd0 = sdesc_sw128(tiles), vd0 = sdesc_n_major(tiles + TILES * TILE, PANEL), qd0 = sdesc_sw128(q_tile);
        int n = 0, item = 0;
#pragma unroll 1
        while (n < chunks && ok) {
            if (!wait(item_full[(unsigned)item % kItems], (unsigned)item / kItems)) break;
            const int count = items[(unsigned)item % kItems].count, steps = PAIR ? 2 * count : count;
            release(item_empty[(unsigned)item % kItems]);
            if (!wait(q_full, item)) break;
#pragma unroll 1
            for (int t = 0; t < steps + 2; ++t) {
                const int x = n + (PAIR ? t >> 1 : t), stream = PAIR ? t & 1 : x & 1;  // of S
                const uint32_t s_at = tmem + stream * kTokens;
                if (t >= 2) {
                    const int y = PAIR ? x - 1 : x - 2, tile = y & (TILES - 1);  // the chunk of O
                    if (!wait(tile_full[2 + tile], y / TILES) || !wait(p_ready[stream], PAIR ? y : y >> 1)) break;
                    tc_fence_after();
                    const uint64_t vd = vd0 + (uint64_t)(tile * (TILE >> 4));
                    const uint32_t o = tmem + kOCol + (ONE ? 0 : stream * 128);
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < kTokens / 16; ++s)
                            mma_ts(o, s_at + 8 * s, vd + (uint64_t)s * (2048 >> 4), idesc_o, t >= (ONE ? 3 : 4) || s > 0);
                        if (!PAIR || stream) mma_commit(smem_u32(&tile_empty[2 + tile]));
                        if constexpr (ONE) mma_commit(smem_u32(&o_added));
                    }
                }
                if (t < steps) {
                    const int tile = x & (TILES - 1);
                    if (!wait(tile_full[tile], x / TILES)) break;
                    tc_fence_after();
                    const uint64_t kd = kd0 + (uint64_t)(tile * (TILE >> 4)), qd = qd0 + (uint64_t)(PAIR ? stream * (TILE >> 4) : 0);
                    auto step = [&](int s) {
                        const uint64_t off = (uint64_t)((s >> 2) * (PANEL >> 4) + (s & 3) * 2);
                        mma_f16_ss(s_at, qd + off, kd + off, idesc_s, s > 0);
                    };
                    if (c.D == DP) {
                        if (elect_one()) {
#pragma unroll
                            for (int s = 0; s < DP / 16; ++s) step(s);
                        }
                    } else {
#pragma unroll 1
                        for (int s = 0; s < c.D / 16; ++s)
                            if (elect_one()) step(s);
                    }
                    if (elect_one()) {
                        mma_commit(smem_u32(&s_full[stream]));
                        if (!PAIR || stream) mma_commit(smem_u32(&tile_empty[tile]));
                    }
                }
            }
            if (ok && elect_one()) mma_commit(smem_u32(&o_full));
            n += count;
            ++item;
        }
        // nothing of this warp's is in flight when the block ends
        if (elect_one()) mma_commit(smem_u32(&mma_end));
        (void)mbar_wait_short(smem_u32(&mma_end), 0, c.status);
        __syncwarp();
    } else {
        // warp 2: scales of K, 3: of V; four tokens a lane, their words asked for a chunk ahead
        const bool is_v = warp == 3;
        float unit[2] = {0.0f, 0.0f};
        int left = 0, item = 0, len = 0, pos = 0, seen_by_all = 0;
        uint32_t apart = 0;  // bit of a stream
        uint4 ahead = make_uint4(0, 0, 0, 0);
        uint32_t ahead_there = 0;
        auto ask = [&](int n) {
            if (!wait(place_full[(unsigned)n % kPlaces], (unsigned)n / kPlaces)) return;
            const int64_t at = places[(unsigned)n % kPlaces][lane / 4].words;
            ahead_there = present[(unsigned)n % kPlaces];
            release(place_empty[(unsigned)n % kPlaces]);
            if (at >= 0)
                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(ahead.x), "=r"(ahead.y), "=r"(ahead.z), "=r"(ahead.w)
                             : "l"(c.pages + at + (is_v ? 4 * c.page : 0) + 16 * (lane & 3)));
        };
#pragma unroll 1
        for (int n = -1; n < chunks && ok; ++n) {
            const int slot = n & (kInfos - 1);
            const uint4 w = ahead;
            const uint32_t there = ahead_there;
            if (n + 1 < chunks) ask(n + 1);
            if (n < 0) continue;
            if (left == 0) {
                if (!wait(item_full[(unsigned)item % kItems], (unsigned)item / kItems)) break;
                const Item &at = items[(unsigned)item % kItems];
                left = at.count, len = at.len, pos = at.chunk * kTokens + 4 * lane;
                const int t_first = min(at.rt * ROWS / a.group, at.T - 1);
                seen_by_all = a.mask ? at.len - at.T : min(at.len, at.len - at.T + t_first + 1);
                apart = 0;
                release(item_empty[(unsigned)item % kItems]);
                ++item;
                unit[0] = unit[1] = pow2i(-126);
            }
            --left;
            Info &info = infos[slot];
            if (n >= kInfos && !wait(info_empty[slot], (unsigned)n / kInfos - 1)) break;
            float s[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
            const int valid = there >> (lane / 4) & 1u ? len - pos : 0;  // beyond the sequence the words are anything
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (U4) s[e] = __uint_as_float(__float_as_uint(s[e]) & 0xffff0000u);
                if (e >= valid) s[e] = 0.0f;
            }
            if (is_v) {
                const int stream = SPLIT ? n & 1 : 0;
                float top = 0.0f, common = 0.0f;  // the largest, and of those that all rows see
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, s[e]), common = pos + e < seen_by_all ? fmaxf(common, s[e]) : common;
                common = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(common)));
                const float old = stream ? unit[1] : unit[0], now = fmaxf(old, pow2_above(common)), per = pow2_inverse(now);
                if (stream) unit[1] = now;
                else unit[0] = now;
                if (__any_sync(0xffffffffu, top > now)) apart |= 1u << stream;
                const bool each = apart >> stream & 1u;
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = each ? s[e] : s[e] * per * (float)(1 << kAttnRoom);
                if (lane == 0) {
                    info.ratio = old * per, info.unit = now, info.before = old;
                    info.present = each ? there | kApart
                                   : there == 0xffu && pos + kTokens <= seen_by_all ? kWhole : there;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] *= a.scale_log2;
            }
            *reinterpret_cast<float2 *>(info.scales[2 * lane] + 2 * is_v) = make_float2(s[0], s[1]);
            *reinterpret_cast<float2 *>(info.scales[2 * lane + 1] + 2 * is_v) = make_float2(s[2], s[3]);
            release(info_full[slot]);
            pos += kTokens;
        }
    }
    } else if (warp < kRowWarp0) {
        regs_dec<128>();
        // Warps 4 and 5 have K, 6 and 7 V, each 64 tokens of a chunk, in registers a chunk ahead.  Eight
        // lanes have four 16-byte pieces of two rows at a time: what they store of a chunk of 8 f16 then
        // lies in eight different places of the swizzle.
        const int is_v = (warp - kCodeWarp0) >> 1, side = warp & 1;
        const int r8 = 2 * (lane >> 3) + (lane >> 2 & 1), quad = lane & 3;
        constexpr int H = U4 ? (DP + 127) / 128 : DP / 64;  // pieces of a row that a lane has
        constexpr int HB = H < 2 ? H : 2, NB = 2 * H / HB;  // pieces, of a chunk's batches, two of which are in registers
        const uint8_t *from[H], *word_from = c.pages + (is_v ? 4 * c.page : 0) + 4 * r8;
        uint32_t to[H];  // of the lane's pieces, in a tile
        bool second[H];
        const uint32_t top = tiles + TILES * is_v * TILE + (64 * side + r8) * 128;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int piece = min(4 * h + quad, c.chunks - 1);  // beyond the row: its last once more
            from[h] = c.pages + (is_v ? c.page * c.row_bytes : 0) + r8 * c.row_bytes + 16 * piece;
            const int chunk = kv_chunk(c.chunks, r8, piece);  // which the piece holds: the order is its own inverse
            // u4: a piece has four chunks of f16; those of every second panel begin with the third of them
            if constexpr (U4) to[h] = top + (chunk >> 1) * PANEL + (((4 * (chunk & 1) + (chunk & 2)) ^ r8) << 4);
            else to[h] = top + (chunk >> 2) * PANEL + (((2 * (chunk & 3)) ^ r8) << 4);
            second[h] = U4 && (chunk & 2);
        }
        uint4 w[2][4][HB];  // two batches: of 32 tokens, 8 of them at a time, HB of a lane's pieces
        uint32_t word[2][4];
        auto ask = [&](int n, int batch) {
            const int u = batch / (H / HB), h0 = batch % (H / HB) * HB;
            const Tile16 *place = places[(unsigned)n % kPlaces] + 4 * side + 2 * u;
            if (c.num_pages == 0) return;  // any codes will do for tiles that are not there, but not from nowhere
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t at = place[k >> 1].rows + (k & 1) * 8 * c.row_bytes;
#pragma unroll
                for (int h = 0; h < HB; ++h) {
                    uint4 &v = w[batch & 1][k][h];
                    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "l"(from[h0 + h] + at));
                }
                if (U4)
                    asm volatile("ld.global.u32 %0, [%1];"
                                 : "=r"(word[batch & 1][k])
                                 : "l"(word_from + max(place[k >> 1].words, (int64_t)0) + (k & 1) * 32));
            }
        };
        if (chunks > 0 && wait(place_full[0], 0)) {
            ask(0, 0);
            ask(0, 1);
            if constexpr (NB == 2) release(place_empty[0]);
        }
#pragma unroll 1
        for (int n = 0; n < chunks && ok; ++n) {
            if (n + 1 < chunks && !wait(place_full[(unsigned)(n + 1) % kPlaces], (unsigned)(n + 1) / kPlaces)) break;
            if (n >= TILES && !wait(tile_empty[2 * is_v + (n & (TILES - 1))], n / TILES - 1)) break;
            const uint32_t tile = (n & (TILES - 1)) * TILE;
#pragma unroll
            for (int batch = 0; batch < NB; ++batch) {
                const int u = batch / (H / HB), h0 = batch % (H / HB) * HB;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const Zero z = zero_of(word[batch & 1][k] & 15u, word[batch & 1][k] & 15u);
                    const uint32_t at = tile + (4 * u + k) * 1024;
#pragma unroll
                    for (int h = 0; h < HB; ++h) {
                        const uint4 v = w[batch & 1][k][h];
                        const uint32_t t = to[h0 + h];
                        const bool swap = second[h0 + h];
                        uint32_t f[4];
                        if constexpr (U4) {
                            u4_pairs(swap ? v.z : v.x, z, f), sts_v4(t + at, f[0], f[1], f[2], f[3]);
                            u4_pairs(swap ? v.w : v.y, z, f), sts_v4((t ^ 16u) + at, f[0], f[1], f[2], f[3]);
                            u4_pairs(swap ? v.x : v.z, z, f), sts_v4((t ^ 32u) + at, f[0], f[1], f[2], f[3]);
                            u4_pairs(swap ? v.y : v.w, z, f), sts_v4((t ^ 48u) + at, f[0], f[1], f[2], f[3]);
                        } else {
                            s8_pairs(v.x, f[0], f[1]), s8_pairs(v.y, f[2], f[3]);
                            sts_v4(t + at, f[0], f[1], f[2], f[3]);
                            s8_pairs(v.z, f[0], f[1]), s8_pairs(v.w, f[2], f[3]);
                            sts_v4((t ^ 16u) + at, f[0], f[1], f[2], f[3]);
                        }
                    }
                }
                if (batch + 2 < NB) ask(n, batch + 2);
                else if (n + 1 < chunks) ask(n + 1, batch + 2 - NB);
                if (NB > 2 && batch + 3 == NB) release(place_empty[(unsigned)n % kPlaces]);
            }
            if (NB == 2 && n + 1 < chunks) release(place_empty[(unsigned)(n + 1) % kPlaces]);
            fence_proxy_async_smem();
            release(tile_full[2 * is_v + (n & (TILES - 1))]);
        }
    } else {
        regs_inc<152>();
        // All eight warps have the streams' steps in turn, while the other stream's products are under way: warps
        // w and w + 4 have 16 rows each of a quarter of them.
        const int part = (warp - kRowWarp0) >> 2, r = (threadIdx.x - kRowWarp0 * 32) & 127;
        const int g = lane >> 2, j = lane & 3;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        auto meet = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        auto all_ok = [&]() {  // of all rows' warps: they wait for each other below, so they leave together
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 p, %1, 0;\n\t"
                "bar.red.and.pred q, 1, 256, p;\n\t"
                "selp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"((uint32_t)ok)
                : "memory");
            return r != 0;
        };
        int n = 0, item = 0;
        while (n < chunks) {
            (void)wait(item_full[(unsigned)item % kItems], (unsigned)item / kItems);
            if (!all_ok()) break;
            const Item &at = items[(unsigned)item % kItems];
            // row0, r: of q and the sums; PAIR: the rows of stream `part`, else all, half of the channels each
            const int count = at.count, row0 = at.rt * ROWS + (PAIR ? part * kRows : 0);
            const int width = min(kRows, at.T * a.group - row0);
            const int rr = row0 + r;
            const bool live = r < width, starts_here = n > 0 || at.chunk == 0, ends_here = at.chunk + count == at.units;
            const int64_t out_row = at.first + rr / a.group;
            const int hq = at.h * a.group + rr % a.group;

            // q: four lanes have a row of the warp's 32, or its half, eight rows at a time; a row's largest value is
            // brought near f16's by a power of two
            {
                constexpr int W = PAIR ? DP / 32 : DP / 64;  // pieces of 8 values of a lane
                const int mine = PAIR ? c.D : c.D / 2;       // a multiple of 16
                const int quad = lane & 3, r0 = 32 * (warp & 3) + (lane >> 2);
                constexpr int E = 2;  // of a lane's four rows at a time
#pragma unroll 1
                for (int e0 = 0; e0 < 4; e0 += E) {
                    uint4 w[E][W];
                    float top[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int row = row0 + r0 + 8 * (e0 + e);
                        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (at.first + row / a.group) * a.ld_q +
                                             (int64_t)(at.h * a.group + row % a.group) * c.D + (PAIR ? 0 : part * mine);
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const int piece = quad + 4 * i;
                            w[e][i] = make_uint4(0, 0, 0, 0);
                            if (r0 + 8 * (e0 + e) < width && 8 * piece < mine)
                                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(w[e][i].x), "=r"(w[e][i].y), "=r"(w[e][i].z), "=r"(w[e][i].w)
                                             : "l"(qp + 8 * piece));
                        }
                    }
                    auto value = [&](uint32_t v, int hi) {
                        const uint32_t h = hi ? v >> 16 : v & 0xffffu;
                        return a.bf16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((uint16_t)h));
                    };
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        top[e] = 0.0f;
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const uint32_t u[4] = {w[e][i].x, w[e][i].y, w[e][i].z, w[e][i].w};
#pragma unroll
                            for (int k = 0; k < 8; ++k) top[e] = fmaxf(top[e], fabsf(value(u[k / 2], k & 1)));
                        }
                        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                        if (!PAIR && quad == 0) row_top[part][r0 + 8 * (e0 + e)] = top[e];
                    }
                    if constexpr (!PAIR) meet();
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int own = r0 + 8 * (e0 + e);
                        const float most = PAIR ? top[e] : fmaxf(row_top[0][own], row_top[1][own]);
                        const RowUnit by(most);
                        if (quad == 0 && (PAIR || part == 0)) row_c[part][own] = by.down;
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const int piece = quad + 4 * i, chunk = (PAIR ? 0 : part * (mine / 8)) + piece;
                            const uint32_t u[4] = {w[e][i].x, w[e][i].y, w[e][i].z, w[e][i].w};
                            uint32_t f[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                // the order in which codes are unpacked: u4 0 4, 1 5, 2 6, 3 7
                                const float lo = U4 ? value(u[x / 2], x & 1) : value(u[x], 0);
                                const float hi = U4 ? value(u[2 + x / 2], x & 1) : value(u[x], 1);
                                const __half2 h = __floats2half2_rn(by.up(lo), by.up(hi));
                                f[x] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            if (8 * piece < mine)
                                sts_v4(q_tile + (PAIR ? part * TILE : 0) + (chunk >> 3) * PANEL + own * 128 +
                                           (((chunk & 7) ^ (own & 7)) << 4),
                                       f[0], f[1], f[2], f[3]);
                        }
                    }
                }
                fence_proxy_async_smem();
                release(q_full);
            }
            meet();
            // of rows q = 0, 1 of this thread, in both streams
            const int own = 32 * (warp & 3) + 16 * part + g, steps = PAIR ? 2 * count : count;
            float cr[2][2], m[2][2], l[2][2], unit[SPLIT ? 2 : 1];  // PAIR: the same of both
            uint32_t apart = 0;  // bit of a stream: its rows' units are in row_unit
#pragma unroll
            for (int st = 0; st < 2; ++st) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    cr[st][q] = row_c[PAIR ? st : 0][own + 8 * q];
                    m[st][q] = -INFINITY;
                    l[st][q] = 0.0f;
                }
                if (st == 0 || SPLIT) unit[st] = pow2i(-126);
            }
            const uint32_t down = (uint32_t)(16 * part) << 16;
            // a warp whose wait gave up goes on to the end of the item: the others wait for it there
#pragma unroll 1
            for (int step = 0; step < steps; ++step) {
                const int i = PAIR ? step >> 1 : step, x = n + i, stream = (PAIR ? step : x) & 1, slot = (unsigned)x % kInfos;
                if (!PAIR || !stream) (void)wait(info_full[slot], (unsigned)x / kInfos);
                (void)wait(s_full[stream], PAIR ? x : x >> 1);
                tc_fence_after();
                const uint32_t there = infos[slot].present;
                const float ratio = infos[slot].ratio;
                uint32_t scales = smem_u32(infos[slot].scales[j]);
                asm volatile("" : "+r"(scales));  // so that no read of them goes ahead of the waits above
                const uint32_t s_at = lanes + down + stream * kTokens, o_at = lanes + down + kOCol + (ONE ? 0 : stream * 128);
                const int own_state = ONE ? 0 : stream;
                auto sums_still = [&]() {  // the others' products are done where S is
                    if constexpr (ONE) {
                        (void)wait(o_added, x - 1);
                        tc_fence_after();
                    }
                };
                // by selection and not by index: the arrays stay in registers
                float sc[2], sm[2], sl[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    sc[q] = own_state ? cr[1][q] : cr[0][q], sm[q] = own_state ? m[1][q] : m[0][q];
                    sl[q] = own_state ? l[1][q] : l[0][q];
                }
                if (there == kWhole) {
                    const uint32_t none[4] = {};
                    weights<false, false, DP>(s_at, o_at, scales, none, j, step < (ONE ? 1 : 2), ratio, sc, sm, sl, nullptr,
                                              sums_still);
                } else {
                    const int pos0 = (at.chunk + i) * kTokens;
                    uint32_t bits[4];
                    const int row = at.rt * ROWS + (PAIR ? stream * kRows : 0) + 32 * (warp & 3) + 16 * part + (lane & 15);
                    const int t = min(row / a.group, at.T - 1);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        bits[w] = seen_bits(a, at, t, pos0 + 32 * w) &
                                  ((there >> (2 * w) & 1u ? 0xffffu : 0u) | (there >> (2 * w + 1) & 1u ? 0xffff0000u : 0u));
                    __syncwarp();
                    if (!(there & kApart)) {
                        weights<true, false, DP>(s_at, o_at, scales, bits, j, step < (ONE ? 1 : 2), ratio, sc, sm, sl, nullptr,
                                                 sums_still);
                    } else {
                        float own_unit[2], *at_unit = &row_unit[own_state][own];
#pragma unroll
                        for (int q = 0; q < 2; ++q) own_unit[q] = apart >> own_state & 1u ? at_unit[8 * q] : infos[slot].before;
                        weights<true, true, DP>(s_at, o_at, scales, bits, j, step < (ONE ? 1 : 2), ratio, sc, sm, sl, own_unit,
                                                sums_still);
                        apart |= 1u << own_state;
                        if (j == 0) at_unit[0] = own_unit[0], at_unit[8] = own_unit[1];
                    }
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (own_state) m[1][q] = sm[q], l[1][q] = sl[q];
                    else m[0][q] = sm[q], l[0][q] = sl[q];
                }
                if (SPLIT && stream) unit[SPLIT ? 1 : 0] = infos[slot].unit;
                else unit[0] = infos[slot].unit;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&p_ready[stream]));
                    if (!PAIR || stream) mbar_arrive(smem_u32(&info_empty[slot]));
                }
            }

            // the row's part of the item: of stream `part`, without PAIR of both streams, 8 channels in turn
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    l[st][q] += __shfl_xor_sync(0xffffffffu, l[st][q], 1);
                    l[st][q] += __shfl_xor_sync(0xffffffffu, l[st][q], 2);
                    if (j == 0) {
                        const int row = own + 8 * q;
                        row_m[st][row] = m[st][q], row_l[st][row] = l[st][q];
                        if (!(apart >> st & 1u)) row_unit[st][row] = unit[SPLIT ? st : 0];
                    }
                }
            (void)wait(o_full, item);
            tc_fence_after();
            meet();
            {
                const int s0 = PAIR ? part : 0, s1 = PAIR ? part : SPLIT;
                const float m0 = row_m[s0][r], m1 = row_m[s1][r], up = fmaxf(m0, m1);
                const float f0 = m0 == up ? 1.0f : ex2(m0 - up), f1 = !SPLIT ? 0.0f : m1 == up ? 1.0f : ex2(m1 - up);
                const float total = !SPLIT ? row_l[s0][r] : __fmaf_rn(row_l[0][r], f0, row_l[1][r] * f1);
                const float u0 = row_unit[s0][r], u1 = row_unit[s1][r], top_unit = fmaxf(u0, u1);  // (s1: s0 without SPLIT)
                const float per = pow2_inverse(top_unit);
                const bool has0 = !SPLIT || count > 1 || !(n & 1), has1 = SPLIT && (count > 1 || (n & 1));
                const float g0 = !SPLIT ? 1.0f : f0 * (u0 * per), g1 = !SPLIT ? 0.0f : f1 * (u1 * per);
                const bool done = starts_here && ends_here;
                const int part_row = PAIR ? part * kRows + r : r;
                float *slot = attn_slot(a, blockIdx.x, starts_here ? 1 : 0, ROWS, DP);
                uint16_t *out = static_cast<uint16_t *>(a.out) + out_row * a.ld_out + (int64_t)hq * c.D;
                const float by = total == 0.0f ? 0.0f : top_unit * kAttnWeightUnit / total;
#pragma unroll 1
                for (int d = PAIR ? 0 : 8 * part; d < c.D; d += PAIR ? 8 : 16) {
                    uint32_t v0[8], v1[8];
                    float v[8];
                    __syncwarp();
                    tmem_ld8(lanes + kOCol + s0 * 128 + d, v0);
                    if constexpr (SPLIT) tmem_ld8(lanes + kOCol + 128 + d, v1);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int at_e = U4 ? 2 * (e & 3) + (e >> 2) : e;  // codes are unpacked 0 4, 1 5, 2 6, 3 7
                        v[e] = has0 ? __uint_as_float(v0[at_e]) * g0 : 0.0f;
                        if constexpr (SPLIT)
                            if (has1) v[e] = __fmaf_rn(__uint_as_float(v1[at_e]), g1, v[e]);
                        if (done) v[e] *= by;
                    }
                    if (!live || !ok) continue;
                    if (done) {
                        *reinterpret_cast<uint4 *>(out + d) = make_uint4(attn_pack(a, v[0], v[1]), attn_pack(a, v[2], v[3]),
                                                                        attn_pack(a, v[4], v[5]), attn_pack(a, v[6], v[7]));
                    } else {
                        float4 *to = reinterpret_cast<float4 *>(slot + part_row * DP + d);
                        to[0] = make_float4(v[0], v[1], v[2], v[3]);
                        to[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
                __syncwarp();
                if (live && ok && (PAIR || part == 0)) {
                    if (done) {
                        if (a.lse) a.lse[out_row * a.heads_q + hq] = attn_lse(up, total);
                    } else {
                        slot[ROWS * DP + 2 * part_row] = up, slot[ROWS * DP + 2 * part_row + 1] = total;
                        slot[ROWS * (DP + 2) + part_row] = top_unit;
                    }
                }
            }
            tc_fence_before();  // O has been read before q_full says so
            const bool stored = all_ok();
            if (stored && threadIdx.x == kRowWarp0 * 32 && starts_here && !ends_here) {
                const int tile0 = at.rt * ROWS;
                attn_record(a, share.block_of(share.from + n - at.chunk + at.units - 1), at.first, tile0,
                            min(ROWS, at.T * a.group - tile0), at.h);
            }
            release(item_empty[(unsigned)item % kItems]);
            n += count;
            ++item;
        }
    }
    if (!ok && lane == 0) atomicOr(c.status, kStatusTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <bool U4, int DP, bool PAIR>
qnn_status launch(KvAttnArgs a, cudaStream_t s)
{
    auto kern = kv_attn_rows_kernel<U4, DP, PAIR>;
    static std::atomic<uint64_t> opted_in{0};
    // one block on an SM, whatever it needs: tensor memory is taken whole (of 227 KB, the static part aside)
    constexpr int kMost = 214 << 10;
    const int need = 1024 + (PAIR ? 6 : DP > 128 ? 3 : 5) * kTokens * DP * 2 + (a.c.batch + 1) * 8;
    if (!opt_in_smem(kern, kMost, opted_in, 100)) return QNN_ERR_CUDA;
    return kv_launch(kern, dim3((unsigned)a.blocks), kThreads, std::max(need, 120 << 10), s, a);
}

}  // namespace

// Two tiles of rows to an item where there are rows for both (and room for the sums of the line beside
// six tiles): a chunk's codes are converted once for both.  One against two, 32 heads on 8, D = 128, us: 8
// sequences of 8192 with 33 tokens (132 rows) 103 / 89, 64 tokens 107 / 103; 32 of 2048 in 4 bits, 40 tokens
// 127 / 105; a single one of 8192, 40 tokens 34 / 33, 64 tokens 34 / 38.
AttnPlan attn_rows_plan(const KvArgs &c, int group)
{
    const bool pair = (int64_t)c.tokens * group > kRows && c.batch <= 2048 && c.D <= 128;
    return {pair ? 2 * kRows : kRows, c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256, std::min(kAttnMaxBlocks, sm_count())};
}

qnn_status launch_attn_rows(const KvAttnArgs &a, const AttnPlan &p, bool u4, cudaStream_t s)
{
    if (p.rows > kRows) {
        if (p.channels == 64) return u4 ? launch<true, 64, true>(a, s) : launch<false, 64, true>(a, s);
        return u4 ? launch<true, 128, true>(a, s) : launch<false, 128, true>(a, s);
    }
    if (p.channels == 64) return u4 ? launch<true, 64, false>(a, s) : launch<false, 64, false>(a, s);
    if (p.channels == 256) return u4 ? launch<true, 256, false>(a, s) : launch<false, 256, false>(a, s);
    return u4 ? launch<true, 128, false>(a, s) : launch<false, 128, false>(a, s);
}

}  // namespace qnn
