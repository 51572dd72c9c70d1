// qnn_kv.cuh -- the cache of keys and values: its pages, the sequences of a call, and the
// checks that its calls share.
#pragma once
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>
#include "qnn_float.cuh"
#include "qnn_internal.h"
#include "qnn_ptx.cuh"

namespace qnn {

constexpr int kKvMaxBatch = 4096, kKvMaxHeads = 1024, kKvMaxLen = 1 << 30;

// A head of a page: K codes [page][row], V codes [page][row], K words [page], V words [page].
// A row is D codes (s8 as q + 128, which a magic number turns into an f16; u4 two a byte, the
// lower channel in the lower half), in 16-byte chunks whose order depends on the token (kv_chunk).
struct KvArgs {
    uint8_t *pages;
    const int32_t *table, *lens, *starts;
    int64_t ld_table, rows, page_bytes;
    int num_pages, batch, tokens;
    int heads, D, page, head_bytes, row_bytes, chunks;  // chunks: of a row
    uint32_t per16, magic16;  // 16-token tiles of a page, and 2^32 / per16 rounded up
    uint32_t *status;
};

// Chunk c of token t's row lies at chunk kv_chunk(t, c): so that the attention's reads of
// shared memory (four even or odd tokens' pairs of chunks, two tokens' four chunks, eight tokens'
// equal chunks at a time) meet no bank twice where rows have 128 or 256 bytes, or twice at most
// where they have 64.
__host__ __device__ __forceinline__ int kv_chunk(int chunks, int t, int c)
{
    if ((chunks & 7) == 0) return c ^ (t & 7) ^ ((t & 1) << 2);
    if (chunks == 4) return c ^ (t >> 1 & 3);
    return c;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 as_f2(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ uint64_t as_u64(float2 v)
{
    uint64_t u;
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(v.x), "f"(v.y));
    return u;
}
__device__ __forceinline__ float2 as_f2(uint64_t u)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(u));
    return v;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_f2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(d);
}

// the largest, NaN aside
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

struct KvSeq {
    int64_t first;  // row of the newest tokens' first
    int T, len;     // T < 0: the sequence is left out
};

__device__ __forceinline__ void kv_bad(const KvArgs &a) { atomicOr(a.status, kStatusBadArg); }

// What the device arrays say of sequence b, checked.
__device__ __forceinline__ KvSeq kv_seq(const KvArgs &a, int b)
{
    KvSeq s;
    const int64_t cap = min(a.ld_table * a.page, (int64_t)kKvMaxLen);
    s.len = *reinterpret_cast<const volatile int32_t *>(a.lens + b);
    s.first = (int64_t)b * a.tokens;
    s.T = a.tokens;
    bool ok = s.len >= 0 && s.len <= cap;
    if (a.starts) {
        const volatile int32_t *st = a.starts;
        const int64_t lo = st[b], hi = st[b + 1];
        ok = ok && lo >= 0 && hi >= lo && hi <= a.rows && hi - lo <= a.tokens;
        s.first = lo;
        s.T = (int)(hi - lo);
    }
    if (!ok) {
        kv_bad(a);
        s.T = -1;
        s.len = 0;
    }
    return s;
}

// Tile / per16 for tiles of positions below 2^31 (per16 <= 16: the rounding of magic16 does not reach a
// quotient), and the rest.
__device__ __forceinline__ int kv_page_index(const KvArgs &a, int tile, int *rest)
{
    const int index = a.per16 == 1 ? tile : (int)__umulhi((uint32_t)tile, a.magic16);
    *rest = tile - index * (int)a.per16;
    return index;
}

// The index-th page of sequence b as it stands in the table, and that page if it is one, or -1.
__device__ __forceinline__ int kv_entry(const KvArgs &a, int b, int index)
{
    return *reinterpret_cast<const volatile int32_t *>(a.table + b * a.ld_table + index);
}
__device__ __forceinline__ int kv_checked(const KvArgs &a, int pg)
{
    if (pg >= 0 && pg < a.num_pages) return pg;
    kv_bad(a);
    return -1;
}
__device__ __forceinline__ int kv_page(const KvArgs &a, int b, int index) { return kv_checked(a, kv_entry(a, b, index)); }

inline int kv_row_bytes(const qnn_kv_geom &g) { return g.kv_dt == QNN_S8 ? g.D : g.D / 2; }

inline bool kv_geom_ok(const qnn_kv_geom *g)
{
    return g && g->heads > 0 && g->heads <= kKvMaxHeads && g->D >= 32 && g->D <= 256 && g->D % 32 == 0 &&
           g->page >= 16 && g->page <= 256 && g->page % 16 == 0 && (g->kv_dt == QNN_S8 || g->kv_dt == QNN_U4);
}

// Checks the geometry and the sequences, in the order that every call reports faults in, and
// fills the arguments (all but the status word).
qnn_status kv_args(const qnn_kv_geom *g, const qnn_kv_seqs *q, KvArgs *a);

// Launches as a programmatic dependent of the kernel before it.
template <typename K, typename... A>
qnn_status kv_launch(K kern, dim3 grid, int threads, int smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        (void)cudaGetLastError();
        return QNN_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace qnn
