// w8a8_sort.hpp -- arguments and launchers of the W8A8 products (gemm_w8a8.hip)
// and of the sorting of tokens by expert (moe_sort.hip).
#pragma once
#include "lowbit_internal.hpp"

namespace lowbit {

// ---------------------------------------------------------------------------
// W8A8 products (gemm_w8a8.hip).  Dense: rows = M tokens, offsets null.  By
// expert: rows sorted by expert, expert e's being [offsets[e], offsets[e + 1]).
// ---------------------------------------------------------------------------
struct W8Args {
    const int8_t *x, *w;                 // [x_rows][K], [E][N][K]
    const float *xs, *ws, *bias;         // [x_rows], [E][N], [N] or null
    void *y;                             // [rows][N], bf16 or fp16
    const int32_t *row_slot, *offsets;   // by expert: slot of each row or null, row ranges
    int rows, N, K, E, x_rows, row_div, y_bf16;
    int splits;                          // dense: K split over this many workgroups,
    int32_t *part;                       // their partial sums [splits][rows][N] here
};
// the activation row that output row r reads; a damaged table reads a wrong
// row, never one outside the matrix
__device__ __forceinline__ int w8a8_source_row(const W8Args &p, int r)
{
    if (p.row_slot == nullptr) return r;
    return min(max(p.row_slot[r], 0) / p.row_div, p.x_rows - 1);
}
// false: more tiles than a launch takes (2^40 outputs or so)
bool gemm_w8a8_fits(int M, int N);
size_t gemm_w8a8_workspace(int M, int N, int K);
hipError_t launch_gemm_w8a8(const W8Args &a, void *ws, hipStream_t s);
hipError_t launch_moe_gemm_w8a8(const W8Args &a, hipStream_t s);

// Tokens sorted by expert and back (moe_sort.hip)
size_t moe_sort_workspace(int slots, int E_local);
hipError_t launch_moe_sort(const int32_t *topk_ids, int slots, int E, const int32_t *expert_map, int E_local,
                           int32_t *row_slot, int32_t *slot_row, int32_t *expert_offsets, void *ws, hipStream_t s);
hipError_t launch_moe_permute(const void *x, const float *x_scale, int T, int top_k, int row_bytes,
                              const int32_t *slot_row, void *xp, float *xp_scale, hipStream_t s);
hipError_t launch_moe_unpermute(const void *yp, int bf16, const float *w, int T, int top_k, int H,
                                const int32_t *slot_row, void *y, hipStream_t s);
hipError_t launch_moe_unpermute_backward(const void *dy, const void *yp, int bf16, const float *w, int T, int top_k,
                                         int H, const int32_t *slot_row, void *dyp, float *dw, hipStream_t s);

}  // namespace lowbit

// Not part of the library's interface: the kernel that a product of these sizes
// (as the entry points accept them) takes, so that a test can name the one it is
// for.  E = 0: dense; gathered: rows of x that row_slot picks from, 0 without it.
// choice: streaming or tiles (1 / 0), rows, channels and waves of a workgroup,
// workgroups that share K.
extern "C" void lowbit_internal_w8a8_choice(int E, int rows, int N, int K, int gathered, int *choice);
