// kv_cache.hpp -- arguments, page layout and launchers of the quantised
// key/value cache (kv_cache.hip: writing and reading; kv_attention.hip).
#pragma once
#include "lowbit_internal.hpp"

namespace lowbit {

typedef uint16_t us8 __attribute__((ext_vector_type(8)));

constexpr int kKvMaxHeads = 1 << 14;

struct KvArgs {
    uint8_t *data;                       // [pages][heads][part]
    const int32_t *table, *len, *offsets;
    int fmt, pages, page_shift, heads, dim;
    int part;                            // bytes of one head in a page
    int width, count, rows, max_rows;    // max_rows <= rows
};

__host__ __device__ constexpr int kv_code_bytes(int fmt, int tokens, int dim)
{
    return fmt == LOWBIT_KV_I8 ? tokens * dim : tokens * dim / 2;
}
// fp32 arrays of a head in a page: scales, and minima for 4 bits
__host__ __device__ constexpr int kv_arrays(int fmt) { return fmt == LOWBIT_KV_I8 ? 2 : 4; }
__host__ __device__ constexpr int kv_part_bytes(int fmt, int page_size, int dim)
{
    return 2 * kv_code_bytes(fmt, page_size, dim) + kv_arrays(fmt) * page_size * 4;
}

// One sequence of a call: its rows and tokens.  Damaged offsets are cut so that
// no row outside the matrices is named.
struct KvSeq {
    int row0, n;                         // first row; rows to work on
    int len;                             // tokens, as the call gives it (not negative)
    int pos0;                            // token that row0 stands for (may be negative)
};
__device__ __forceinline__ KvSeq kv_sequence(const KvArgs &a, int b)
{
    KvSeq s;
    const int at = min(max(a.offsets[b], 0), a.rows), end = min(max(a.offsets[b + 1], at), a.rows);
    s.row0 = at;
    s.n = min(end - at, a.max_rows);
    s.len = max(a.len[b], 0);
    s.pos0 = s.len - (end - at);
    return s;
}
// page of tokens [64 * block, +64) of sequence b, or -1
__device__ __forceinline__ int kv_page(const KvArgs &a, int b, int block)
{
    const int i = block >> (a.page_shift - 6);
    if (i < 0 || i >= a.width) return -1;
    const int page = a.table[(int64_t)b * a.width + i];
    return page >= 0 && page < a.pages ? page : -1;
}
__device__ __forceinline__ uint8_t *kv_part(const KvArgs &a, int page, int head)
{
    return a.data + ((int64_t)page * a.heads + head) * a.part;
}

// Blocks of 64 tokens that `rows` tokens in a row can touch
constexpr int kv_blocks(int rows) { return (int)(((int64_t)rows + 62) / 64 + 1); }
inline bool kv_rows_fit(const KvArgs &a)
{
    return (int64_t)a.count * kv_blocks(a.max_rows) * 2 * a.heads < ((int64_t)1 << 24);
}

hipError_t launch_kv_write(const KvArgs &a, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int bf16,
                           hipStream_t s);
hipError_t launch_kv_read(const KvArgs &a, void *k, int64_t k_stride, void *v, int64_t v_stride, int bf16,
                          hipStream_t s);

bool kv_attention_fits(const KvArgs &a, int q_heads);
size_t kv_attention_workspace(const KvArgs &a, int q_heads);
hipError_t launch_kv_attention(const KvArgs &a, const void *q, int64_t q_stride, int q_heads, int bf16, float scale,
                               int window, void *y, void *ws, hipStream_t s);

}  // namespace lowbit
