// moe_sort.hip -- tokens sorted by expert and back: the index that sorts the
// routed slots, the tokens' rows brought into that order, the rows summed back
// into token order with the router's weights, and the gradient of that sum.
//
// Slot s = t * top_k + j is token t's j-th routed expert.  Its key is the local
// number of that expert; a slot whose key is outside [0, E_local) has no row.
//   slot_row[s]  = #{s' : key(s') < key(s)} + #{s' < s : key(s') = key(s)},  -1 without a row
//   permute      : xp[slot_row[s]] = x[t]
//   unpermute    : y[t] = RNE( sum_j w[t][j] * yp[slot_row[t][j]] )
//   its gradient : dyp[slot_row[s]] = RNE( w[s] * dy[t] ),  dw[s] = sum_h dy[t][h] * yp[slot_row[s]][h]
// The gradient of permute is unpermute without weights (each token's copies
// added up).  Nothing is added with atomics: every output has one writer and a
// fixed order of summation, in fp32.
#include "lowbit_internal.hpp"

namespace lowbit {

namespace {

// ---------------------------------------------------------------- index
// A stable counting sort.  A workgroup of 16 waves takes one chunk of slots,
// each wave a run of it.  Counts per (wave, key) in LDS give, scanned over
// keys, chunks and waves, the first row of every (wave, key); a wave then walks
// its run 64 slots at a time, where a slot's rank among the equal keys of the
// 64 comes from ballots over the key's bits.  One workgroup is the whole sort
// for few slots; for many, a first kernel writes every chunk's histogram and
// each workgroup of the second one sums those of the chunks before its own.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortOneChunk = 8192;              // slots up to which one workgroup sorts
constexpr int kSortMaxChunks = 128;

struct SortArgs {
    const int32_t *ids, *map;
    int32_t *row_slot, *slot_row, *offsets, *hist;
    int slots, E, E_local, chunk, bits;
};

__device__ __forceinline__ int sort_key(const SortArgs &p, int s)
{
    const int id = p.ids[s];
    if (id < 0 || id >= p.E) return -1;
    const int k = p.map ? p.map[id] : id;
    return k >= 0 && k < p.E_local ? k : -1;
}

__global__ __launch_bounds__(kSortThreads) void moe_sort_hist_kernel(SortArgs p)
{
    __shared__ int count[1024];
    const int tid = threadIdx.x;
    count[tid] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(begin + p.chunk, (int64_t)p.slots);
    for (int64_t s = begin + tid; s < end; s += kSortThreads) {
        const int k = sort_key(p, (int)s);
        if (k >= 0) atomicAdd(&count[k], 1);
    }
    __syncthreads();
    if (tid < p.E_local) p.hist[(int64_t)blockIdx.x * p.E_local + tid] = count[tid];
}

// ONE: a single workgroup, no histograms
template <bool ONE>
__global__ __launch_bounds__(kSortThreads) void moe_sort_kernel(SortArgs p)
{
    extern __shared__ int first[];               // [waves][E_local]: counts, then first rows
    __shared__ int before[kSortThreads], total[kSortThreads], wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int El = p.E_local, run = p.chunk / kSortWaves;
    const int64_t base = (int64_t)blockIdx.x * p.chunk + (int64_t)wave * run;
    const int n = (int)min((int64_t)run, max((int64_t)0, (int64_t)p.slots - base));

    for (int i = tid; i < kSortWaves * El; i += kSortThreads) first[i] = 0;
    __syncthreads();
    for (int i = lane; i < n; i += 64) {
        const int k = sort_key(p, (int)(base + i));
        if (k >= 0) atomicAdd(&first[wave * El + k], 1);
    }
    __syncthreads();

    // slots of key tid in all chunks, and in the chunks before this one
    int sum = 0, pre = 0;
    if constexpr (ONE) {
        if (tid < El)
            for (int w = 0; w < kSortWaves; ++w) sum += first[w * El + tid];
    } else {
        // groups of 2^bits threads share the chunks out
        const int width = 1 << p.bits, groups = kSortThreads >> p.bits;
        const int k = tid & (width - 1), g = tid >> p.bits;
        int s = 0, b = 0;
        if (k < El)
#pragma unroll 4
            for (int c = g; c < (int)gridDim.x; c += groups) {
                const int h = p.hist[(int64_t)c * El + k];
                s += h;
                b += c < (int)blockIdx.x ? h : 0;
            }
        total[tid] = s;
        before[tid] = b;
        __syncthreads();
        if (tid < El)
            for (int q = 0; q < groups; ++q) {
                sum += total[(q << p.bits) + tid];
                pre += before[(q << p.bits) + tid];
            }
    }
    // exclusive scan over the keys
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int start = incl - sum, rows = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        start += w < wave ? wave_sum[w] : 0;
        rows += wave_sum[w];
    }
    if (tid < El) {
        if (blockIdx.x == 0) p.offsets[tid] = start;
        int at = start + pre;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = first[w * El + tid];
            first[w * El + tid] = at;
            at += c;
        }
    }
    if (blockIdx.x == 0 && tid == 0) p.offsets[El] = rows;
    __syncthreads();

    for (int i0 = 0; i0 < n; i0 += 64) {
        const int s = (int)(base + i0 + lane);
        const bool in = i0 + lane < n;
        const int k = in ? sort_key(p, s) : -1;
        uint64_t same = __ballot(k >= 0);
        for (int b = 0; b < p.bits; ++b) {
            const uint64_t set = __ballot((k >> b) & 1);
            same &= (k >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
        int at = 0;
        if (k >= 0 && rank == 0) at = atomicAdd(&first[wave * El + k], __popcll(same));
        at = __shfl(at, k >= 0 ? __ffsll((unsigned long long)same) - 1 : lane) + rank;
        if (in) {
            p.slot_row[s] = k >= 0 ? at : -1;
            if (k >= 0) p.row_slot[at] = s;
        }
    }
    // behind the last row
    for (int64_t r = rows + (int64_t)blockIdx.x * kSortThreads + tid; r < p.slots; r += (int64_t)gridDim.x * kSortThreads)
        p.row_slot[r] = p.slots;
}

struct SortPlan {
    int chunk, chunks;
};
SortPlan sort_plan(int slots)
{
    SortPlan pl;
    if (slots <= kSortOneChunk) {
        pl.chunk = (int)round_up(slots > 0 ? slots : 1, kSortThreads);
        pl.chunks = 1;
        return pl;
    }
    const int64_t least = 4 * kSortThreads;
    const int64_t even = round_up(((int64_t)slots + kSortMaxChunks - 1) / kSortMaxChunks, kSortThreads);
    pl.chunk = (int)(even > least ? even : least);
    pl.chunks = (int)(((int64_t)slots + pl.chunk - 1) / pl.chunk);
    return pl;
}

// ---------------------------------------------------------------- rows
// One token per group of `1 << shift` threads (a group walks its token's row
// in 16-byte steps), 256 / group tokens per workgroup.
constexpr int kRowThreads = 256;

// log2 of the threads that share a row of `items`
int row_shift(int64_t items)
{
    int s = 3;
    while (s < 8 && (1 << s) < items) ++s;
    return s;
}

template <typename V>
__global__ __launch_bounds__(kRowThreads)
void moe_permute_kernel(const V *x, const float *x_scale, int T, int top_k, int items, int shift,
                        const int32_t *slot_row, V *xp, float *xp_scale)
{
    const int64_t t = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= T) return;
    const int32_t *rows = slot_row + t * top_k;
    const int64_t limit = (int64_t)T * top_k;
    const int c0 = threadIdx.x & ((1 << shift) - 1);
    for (int c = c0; c < items; c += 1 << shift) {
        const V v = x[t * items + c];
        for (int j = 0; j < top_k; ++j) {
            const int r = rows[j];
            if (r >= 0 && r < limit) xp[(int64_t)r * items + c] = v;
        }
    }
    if (x_scale != nullptr && c0 == 0) {
        const float v = x_scale[t];
        for (int j = 0; j < top_k; ++j) {
            const int r = rows[j];
            if (r >= 0 && r < limit) xp_scale[r] = v;
        }
    }
}

template <bool BF16> struct Elem;
template <> struct Elem<true> { typedef __bf16 v8 __attribute__((ext_vector_type(8))); typedef __bf16 t; };
template <> struct Elem<false> { typedef _Float16 v8 __attribute__((ext_vector_type(8))); typedef _Float16 t; };

template <bool BF16>
__global__ __launch_bounds__(kRowThreads)
void moe_unpermute_kernel(const typename Elem<BF16>::v8 *yp, const float *w, int T, int top_k, int items, int shift,
                          const int32_t *slot_row, typename Elem<BF16>::v8 *y)
{
    typedef typename Elem<BF16>::v8 v8;
    typedef typename Elem<BF16>::t T1;
    const int64_t t = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= T) return;
    const int32_t *rows = slot_row + t * top_k;
    const int64_t limit = (int64_t)T * top_k;
    for (int c = threadIdx.x & ((1 << shift) - 1); c < items; c += 1 << shift) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < top_k; ++j) {
            const int r = rows[j];
            if (r < 0 || r >= limit) continue;
            const float wj = w ? w[t * top_k + j] : 1.f;
            const v8 v = yp[(int64_t)r * items + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(wj, (float)v[i], acc[i]);
        }
        v8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (T1)acc[i];
        y[t * items + c] = o;
    }
}

// One workgroup per token
template <bool BF16>
__global__ __launch_bounds__(kRowThreads)
void moe_unpermute_backward_kernel(const typename Elem<BF16>::v8 *dy, const typename Elem<BF16>::v8 *yp,
                                   const float *w, int T, int top_k, int items, const int32_t *slot_row,
                                   typename Elem<BF16>::v8 *dyp, float *dw)
{
    typedef typename Elem<BF16>::v8 v8;
    typedef typename Elem<BF16>::t T1;
    __shared__ float part[kRowThreads / 64];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int j = 0; j < top_k; ++j) {
        const int64_t s = t * top_k + j;
        const int r = slot_row[s];
        const bool has = r >= 0 && r < (int64_t)T * top_k;
        const float wj = w[s];
        float dot = 0.f;
        if (has)
            for (int c = tid; c < items; c += kRowThreads) {
                const v8 g = dy[t * items + c], v = yp[(int64_t)r * items + c];
                v8 o;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot = __builtin_fmaf((float)g[i], (float)v[i], dot);
                    o[i] = (T1)(wj * (float)g[i]);
                }
                dyp[(int64_t)r * items + c] = o;
            }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
        if (lane == 0) part[wave] = dot;
        __syncthreads();
        if (tid == 0) dw[s] = has ? (part[0] + part[1]) + (part[2] + part[3]) : 0.f;
        __syncthreads();
    }
}

}  // namespace

size_t moe_sort_workspace(int slots, int E_local)
{
    const SortPlan pl = sort_plan(slots);
    return pl.chunks > 1 ? (size_t)pl.chunks * E_local * sizeof(int32_t) : 0;
}

hipError_t launch_moe_sort(const int32_t *topk_ids, int slots, int E, const int32_t *expert_map, int E_local,
                           int32_t *row_slot, int32_t *slot_row, int32_t *expert_offsets, void *ws, hipStream_t s)
{
    const SortPlan pl = sort_plan(slots);
    int bits = 1;
    while ((1 << bits) < E_local) ++bits;
    const SortArgs a = {topk_ids, expert_map, row_slot, slot_row, expert_offsets, static_cast<int32_t *>(ws),
                        slots, E, E_local, pl.chunk, bits};
    const size_t lds = (size_t)kSortWaves * E_local * sizeof(int);
    if (pl.chunks == 1) {
        moe_sort_kernel<true><<<1, kSortThreads, lds, s>>>(a);
    } else {
        moe_sort_hist_kernel<<<pl.chunks, kSortThreads, 0, s>>>(a);
        moe_sort_kernel<false><<<pl.chunks, kSortThreads, lds, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_moe_permute(const void *x, const float *x_scale, int T, int top_k, int row_bytes,
                              const int32_t *slot_row, void *xp, float *xp_scale, hipStream_t s)
{
    const bool wide = row_bytes % 16 == 0;
    const int items = row_bytes / (wide ? 16 : 8), shift = row_shift(items);
    const unsigned blocks = (unsigned)(((int64_t)T + (256 >> shift) - 1) >> (8 - shift));
    if (wide)
        moe_permute_kernel<u4><<<blocks, kRowThreads, 0, s>>>(static_cast<const u4 *>(x), x_scale, T, top_k, items,
                                                              shift, slot_row, static_cast<u4 *>(xp), xp_scale);
    else
        moe_permute_kernel<uint2><<<blocks, kRowThreads, 0, s>>>(static_cast<const uint2 *>(x), x_scale, T, top_k,
                                                                 items, shift, slot_row, static_cast<uint2 *>(xp),
                                                                 xp_scale);
    return hipGetLastError();
}

namespace {
template <bool BF16>
void unpermute(const void *yp, const float *w, int T, int top_k, int items, const int32_t *slot_row, void *y,
               hipStream_t s)
{
    typedef typename Elem<BF16>::v8 v8;
    const int shift = row_shift(items);
    const unsigned blocks = (unsigned)(((int64_t)T + (256 >> shift) - 1) >> (8 - shift));
    moe_unpermute_kernel<BF16><<<blocks, kRowThreads, 0, s>>>(static_cast<const v8 *>(yp), w, T, top_k, items, shift,
                                                              slot_row, static_cast<v8 *>(y));
}
template <bool BF16>
void unpermute_backward(const void *dy, const void *yp, const float *w, int T, int top_k, int items,
                        const int32_t *slot_row, void *dyp, float *dw, hipStream_t s)
{
    typedef typename Elem<BF16>::v8 v8;
    moe_unpermute_backward_kernel<BF16><<<(unsigned)T, kRowThreads, 0, s>>>(
        static_cast<const v8 *>(dy), static_cast<const v8 *>(yp), w, T, top_k, items, slot_row, static_cast<v8 *>(dyp),
        dw);
}
}  // namespace

hipError_t launch_moe_unpermute(const void *yp, int bf16, const float *w, int T, int top_k, int H,
                                const int32_t *slot_row, void *y, hipStream_t s)
{
    if (bf16)
        unpermute<true>(yp, w, T, top_k, H / 8, slot_row, y, s);
    else
        unpermute<false>(yp, w, T, top_k, H / 8, slot_row, y, s);
    return hipGetLastError();
}

hipError_t launch_moe_unpermute_backward(const void *dy, const void *yp, int bf16, const float *w, int T, int top_k,
                                         int H, const int32_t *slot_row, void *dyp, float *dw, hipStream_t s)
{
    if (bf16)
        unpermute_backward<true>(dy, yp, w, T, top_k, H / 8, slot_row, dyp, dw, s);
    else
        unpermute_backward<false>(dy, yp, w, T, top_k, H / 8, slot_row, dyp, dw, s);
    return hipGetLastError();
}

}  // namespace lowbit
