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
#include <algorithm>
#include <type_traits>

#include "w8a8_sort.hpp"

namespace lowbit {

namespace {

// ---------------------------------------------------------------- index
// A stable counting sort.  A workgroup of 16 waves takes one chunk of slots,
// each wave a run of it, 64 slots at a time.  A slot's rank among the equal
// keys of the 64 comes from ballots over the key's bits, and one LDS add per
// key and 64 slots gives its place among the wave's; those counts, scanned over
// keys, chunks and waves, give the first row of every (wave, key).  One
// workgroup is the whole sort for few slots; for many, a first kernel writes
// every chunk's histogram and each workgroup of the second one sums those of
// the chunks before its own.  All of it is latency: 296 slots in 2.9 us (an
// empty launch takes 2.2), 131072 in 4.8 + 5.7 us where their bytes take 0.3.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortOneChunk = 8192;              // slots up to which one workgroup sorts
constexpr int kSortMaxChunks = 128;
constexpr int kSortKept = 8;                     // slots a thread keeps in registers, at most

struct SortArgs {
    const int32_t *ids, *map;
    int32_t *row_slot, *slot_row, *offsets, *hist;
    int slots, E, E_local, chunk, bits;
};

__device__ __forceinline__ int sort_key(const SortArgs &p, int64_t s)
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
        const int k = sort_key(p, s);
        if (k >= 0) atomicAdd(&count[k], 1);
    }
    __syncthreads();
    if (tid < p.E_local) p.hist[(int64_t)blockIdx.x * p.E_local + tid] = count[tid];
}

// The place of the lane's slot among those of its key that the wave has met: `met` counts them by key
__device__ __forceinline__ int sort_place(int k, int bits, int *met)
{
    const int lane = threadIdx.x & 63;
    uint64_t same = __ballot(k >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((k >> b) & 1);
        same &= (k >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
    int at = 0;
    if (k >= 0 && rank == 0) at = atomicAdd(&met[k], __popcll(same));
    return __shfl(at, k >= 0 ? __ffsll((unsigned long long)same) - 1 : lane) + rank;
}

// ONE: a single workgroup, no histograms.  R: rounds of 64 slots that a wave
// has at most, keys and places kept in registers; 0: any number, read twice.
template <bool ONE, int R>
__global__ __launch_bounds__(kSortThreads) void moe_sort_kernel(SortArgs p)
{
    extern __shared__ int first[];               // [waves][E_local]: counts, then first rows
    __shared__ int before[kSortThreads], total[kSortThreads], wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int El = p.E_local, run = p.chunk / kSortWaves;
    const int64_t base = (int64_t)blockIdx.x * p.chunk + (int64_t)wave * run;
    const int n = (int)min((int64_t)run, max((int64_t)0, (int64_t)p.slots - base));
    constexpr int KEPT = R > 0 ? R : 1;
    int key[KEPT], place[KEPT];

    if constexpr (R > 0)
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = i * 64 + lane < n ? sort_key(p, base + i * 64 + lane) : -1;
    int sum = 0, pre = 0;
    if constexpr (!ONE) {
        // slots of each key in all chunks and in those before this one: groups of 2^bits threads share the chunks
        const int groups = kSortThreads >> p.bits;
        const int k = tid & ((1 << p.bits) - 1);
        int s = 0, b = 0;
        if (k < El)
#pragma unroll 8
            for (int c = tid >> p.bits; c < (int)gridDim.x; c += groups) {
                const int h = p.hist[(int64_t)c * El + k];
                s += h;
                b += c < (int)blockIdx.x ? h : 0;
            }
        total[tid] = s;
        before[tid] = b;
    }
    for (int i = tid; i < kSortWaves * El; i += kSortThreads) first[i] = 0;
    __syncthreads();
    if constexpr (!ONE) {
        if (tid < El)
            for (int q = tid; q < kSortThreads; q += 1 << p.bits) {
                sum += total[q];
                pre += before[q];
            }
    }
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i * 64 < n) place[i] = sort_place(key[i], p.bits, first + wave * El);
    } else {
        for (int i = lane; i < n; i += 64) {
            const int k = sort_key(p, base + i);
            if (k >= 0) atomicAdd(&first[wave * El + k], 1);
        }
    }
    __syncthreads();

    int count[kSortWaves];
    if (tid < El)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) count[w] = first[w * El + tid];
    if constexpr (ONE) {
        if (tid < El)
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) sum += count[w];
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
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        start += w < wave ? wave_sum[w] : 0;
        rows += wave_sum[w];
    }
    if (tid < El) {
        if (blockIdx.x == 0) p.offsets[tid] = start;
        int at = start + pre;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            first[w * El + tid] = at;
            at += count[w];
        }
    }
    if (blockIdx.x == 0 && tid == 0) p.offsets[El] = rows;
    __syncthreads();

    auto put = [&](int i, int k, int at) __attribute__((always_inline)) {
        p.slot_row[base + i] = k >= 0 ? at : -1;
        if (k >= 0) p.row_slot[at] = (int32_t)(base + i);
    };
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i * 64 + lane < n) put(i * 64 + lane, key[i], key[i] >= 0 ? first[wave * El + key[i]] + place[i] : -1);
    } else {
        for (int i0 = 0; i0 < n; i0 += 64) {
            const bool in = i0 + lane < n;
            const int k = in ? sort_key(p, base + i0 + lane) : -1;
            const int at = sort_place(k, p.bits, first + wave * El);
            if (in) put(i0 + lane, k, at);
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
    const int64_t n = slots > 0 ? slots : 1;
    SortPlan pl;
    pl.chunk = (int)round_up(n <= kSortOneChunk ? n : (n + kSortMaxChunks - 1) / kSortMaxChunks, kSortThreads);
    pl.chunks = (int)((n + pl.chunk - 1) / pl.chunk);
    return pl;
}

typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- rows
// One token per group of `1 << shift` threads (a group walks its token's row
// in 16-byte steps), 256 / group tokens per workgroup.  Bound by the bytes:
// every row is read once and written once, by the token's threads, so that a
// token's row comes from memory once for all its slots.  Rows of 4 KiB: permute
// of 16384 tokens to 131072 rows 100 to 105 us (5.8 to 6.0 TB/s), unpermute of
// 8192 tokens from 49000 rows 41 us (5.7 TB/s), the gradient of 8192 with 65536
// rows 105 to 108 us (5.3 TB/s).
constexpr int kRowThreads = 256;

// log2 of the threads that share a row of `items`
int row_shift(int64_t items)
{
    int s = 3;
    while (s < 8 && (1 << s) < items) ++s;
    return s;
}

// Workgroups along a row: one for each of its steps where the rows are few, as nothing else hides a step's latency
// (permute / unpermute, us: 64 tokens with 2 rows of 16 KiB 3.8 / 5.1 -> 2.8 / 2.9, 333 with 2 of 8 KiB 3.9 / 4.5 ->
// 3.8 / 3.7); one for all where they are many (8192 with 2 of 8 KiB: 43 / 37, 43 / 40 with two).
unsigned row_blocks(int items, int shift, bool far)
{
    return far ? 1 : (unsigned)std::max(1, std::min((items + (1 << shift) - 1) >> shift, 1024));
}

// Rows that no cache will hold until they are used go past it.  Measured at
// 65536 rows of 4 KiB (us, plain / past the caches): permute 59 / 51, unpermute
// 58 / 50, its gradient 111 / 99.
constexpr int64_t kFarBytes = (int64_t)32 << 20;     // the L2 caches of the eight XCDs

template <bool FAR, typename V>
__device__ __forceinline__ V get_row(const V *p)
{
    if constexpr (FAR) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool FAR, typename V>
__device__ __forceinline__ void put_row(V *p, V v)
{
    if constexpr (FAR) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// Slots whose rows a thread has under way together
constexpr int kRowBatch = 8;

// rows of slots j0 .. j0 + kRowBatch - 1 of a token, -1 where there is none
__device__ __forceinline__ void batch_rows(const int32_t *rows, int j0, int top_k, int64_t limit, int (&r)[kRowBatch])
{
#pragma unroll
    for (int j = 0; j < kRowBatch; ++j) r[j] = rows[min(j0 + j, top_k - 1)];
#pragma unroll
    for (int j = 0; j < kRowBatch; ++j)
        if (j0 + j >= top_k || r[j] >= limit) r[j] = -1;
}

template <bool FAR, typename V>
__global__ __launch_bounds__(kRowThreads)
void moe_permute_kernel(const V *x, const float *x_scale, int T, int top_k, int items, int shift,
                        const int32_t *slot_row, V *xp, float *xp_scale)
{
    const int64_t t = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= T) return;
    const int c0 = (blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1)), step = gridDim.y << shift;
    const bool scaled = x_scale != nullptr && c0 == 0;
    const float scale = scaled ? x_scale[t] : 0.f;
    for (int j0 = 0; j0 < top_k; j0 += kRowBatch) {
        int r[kRowBatch];
        batch_rows(slot_row + t * top_k, j0, top_k, (int64_t)T * top_k, r);
        for (int c = c0; c < items; c += step) {
            const V v = x[t * items + c];
#pragma unroll
            for (int j = 0; j < kRowBatch; ++j)
                if (r[j] >= 0) put_row<FAR>(xp + (int64_t)r[j] * items + c, v);
        }
        if (scaled)
#pragma unroll
            for (int j = 0; j < kRowBatch; ++j)
                if (r[j] >= 0) xp_scale[r[j]] = scale;
    }
}

template <bool BF16> struct Elem;
template <> struct Elem<true> { typedef __bf16 v8 __attribute__((ext_vector_type(8))); typedef __bf16 t; };
template <> struct Elem<false> { typedef _Float16 v8 __attribute__((ext_vector_type(8))); typedef _Float16 t; };

template <bool FAR, bool BF16>
__global__ __launch_bounds__(kRowThreads)
void moe_unpermute_kernel(const typename Elem<BF16>::v8 *yp, const float *w, int T, int top_k, int items, int shift,
                          const int32_t *slot_row, typename Elem<BF16>::v8 *y)
{
    typedef typename Elem<BF16>::v8 v8;
    typedef typename Elem<BF16>::t T1;
    const int64_t t = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= T) return;
    const int step = gridDim.y << shift;
    for (int c = (blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1)); c < items; c += step) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < top_k; j0 += kRowBatch) {
            int r[kRowBatch];
            v8 v[kRowBatch];
            batch_rows(slot_row + t * top_k, j0, top_k, (int64_t)T * top_k, r);
#pragma unroll
            for (int j = 0; j < kRowBatch; ++j)
                if (r[j] >= 0) v[j] = get_row<FAR>(yp + (int64_t)r[j] * items + c);
#pragma unroll
            for (int j = 0; j < kRowBatch; ++j)
                if (r[j] >= 0) {
                    const float wj = w ? w[t * top_k + j0 + j] : 1.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(wj, (float)v[j][i], acc[i]);
                }
        }
        v8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (T1)acc[i];
        y[t * items + c] = o;
    }
}

// One workgroup of NW waves per token, kRowBatch slots at a time: their rows are read and written in one pass over
// dy, and their sums cross the lanes together.
template <bool FAR, bool BF16, int NW>
__global__ __launch_bounds__(NW * 64)
void moe_unpermute_backward_kernel(const typename Elem<BF16>::v8 *dy, const typename Elem<BF16>::v8 *yp,
                                   const float *w, int T, int top_k, int items, const int32_t *slot_row,
                                   typename Elem<BF16>::v8 *dyp, float *dw)
{
    typedef typename Elem<BF16>::v8 v8;
    typedef typename Elem<BF16>::t T1;
    __shared__ float part[NW][kRowBatch];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int j0 = 0; j0 < top_k; j0 += kRowBatch) {
        int r[kRowBatch];
        float wj[kRowBatch], dot[kRowBatch];
        batch_rows(slot_row + t * top_k, j0, top_k, (int64_t)T * top_k, r);
#pragma unroll
        for (int j = 0; j < kRowBatch; ++j) {
            wj[j] = w[t * top_k + min(j0 + j, top_k - 1)];
            dot[j] = 0.f;
        }
        for (int c = tid; c < items; c += NW * 64) {
            const v8 g = dy[t * items + c];
            v8 v[kRowBatch];
#pragma unroll
            for (int j = 0; j < kRowBatch; ++j)
                if (r[j] >= 0) v[j] = get_row<FAR>(yp + (int64_t)r[j] * items + c);
#pragma unroll
            for (int j = 0; j < kRowBatch; ++j)
                if (r[j] >= 0) {
                    v8 o;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[j] = __builtin_fmaf((float)g[i], (float)v[j][i], dot[j]);
                        o[i] = (T1)(wj[j] * (float)g[i]);
                    }
                    put_row<FAR>(dyp + (int64_t)r[j] * items + c, o);
                }
        }
        if (j0 > 0) __syncthreads();                  // the sums of the slots before are read
#pragma unroll
        for (int j = 0; j < kRowBatch; ++j) {
            if (j0 + j >= top_k) break;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o);
            if (lane == 0) part[wave][j] = dot[j];
        }
        __syncthreads();
        if (tid < kRowBatch && j0 + tid < top_k) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < NW; ++q) s += part[q][tid];
            dw[t * top_k + j0 + tid] = s;
        }
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
    auto launch = [&](auto kernel) {
        if (E_local > 800) {                          // with the fixed arrays more than 64 KiB: asked for
            const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                     (int)lds);
            if (e != hipSuccess) return e;
        }
        kernel<<<pl.chunks, kSortThreads, lds, s>>>(a);
        return hipGetLastError();
    };
    if (pl.chunks > 1) {
        moe_sort_hist_kernel<<<pl.chunks, kSortThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int rounds = pl.chunk / kSortThreads;
    if (pl.chunks == 1) return rounds == 1 ? launch(moe_sort_kernel<true, 1>) : launch(moe_sort_kernel<true, kSortKept>);
    if (rounds == 1) return launch(moe_sort_kernel<false, 1>);
    return rounds <= kSortKept ? launch(moe_sort_kernel<false, kSortKept>) : launch(moe_sort_kernel<false, 0>);
}

hipError_t launch_moe_permute(const void *x, const float *x_scale, int T, int top_k, int row_bytes,
                              const int32_t *slot_row, void *xp, float *xp_scale, hipStream_t s)
{
    const bool wide = row_bytes % 16 == 0, far = (int64_t)T * top_k * row_bytes > kFarBytes;
    const int items = row_bytes / (wide ? 16 : 8), shift = row_shift(items);
    const unsigned blocks = (unsigned)(((int64_t)T + (256 >> shift) - 1) >> (8 - shift));
    auto launch = [&](auto kernel, auto item) {
        typedef decltype(item) V;
        kernel<<<dim3(blocks, row_blocks(items, shift, far)), kRowThreads, 0, s>>>(static_cast<const V *>(x), x_scale, T, top_k, items, shift, slot_row,
                                              static_cast<V *>(xp), xp_scale);
        return hipGetLastError();
    };
    if (wide) return far ? launch(moe_permute_kernel<true, u4>, u4{}) : launch(moe_permute_kernel<false, u4>, u4{});
    return far ? launch(moe_permute_kernel<true, u2>, u2{}) : launch(moe_permute_kernel<false, u2>, u2{});
}

hipError_t launch_moe_unpermute(const void *yp, int bf16, const float *w, int T, int top_k, int H,
                                const int32_t *slot_row, void *y, hipStream_t s)
{
    const bool far = (int64_t)T * top_k * H * 2 > kFarBytes;
    const int items = H / 8, shift = row_shift(items);
    const unsigned blocks = (unsigned)(((int64_t)T + (256 >> shift) - 1) >> (8 - shift));
    auto launch = [&](auto kernel, auto item) {
        typedef decltype(item) v8;
        kernel<<<dim3(blocks, row_blocks(items, shift, far)), kRowThreads, 0, s>>>(static_cast<const v8 *>(yp), w, T, top_k, items, shift, slot_row,
                                              static_cast<v8 *>(y));
        return hipGetLastError();
    };
    typedef Elem<true>::v8 b8;
    if (bf16) return far ? launch(moe_unpermute_kernel<true, true>, b8{}) : launch(moe_unpermute_kernel<false, true>, b8{});
    return far ? launch(moe_unpermute_kernel<true, false>, h8{}) : launch(moe_unpermute_kernel<false, false>, h8{});
}

hipError_t launch_moe_unpermute_backward(const void *dy, const void *yp, int bf16, const float *w, int T, int top_k,
                                         int H, const int32_t *slot_row, void *dyp, float *dw, hipStream_t s)
{
    const bool far = (int64_t)T * top_k * H * 2 > kFarBytes;
    const int items = H / 8;
    auto launch = [&](auto kernel, int waves, auto item) {
        typedef decltype(item) v8;
        kernel<<<(unsigned)T, waves * 64, 0, s>>>(static_cast<const v8 *>(dy), static_cast<const v8 *>(yp), w, T, top_k,
                                                  items, slot_row, static_cast<v8 *>(dyp), dw);
        return hipGetLastError();
    };
    auto pick = [&](auto b, auto item) {
        constexpr bool B = decltype(b)::value;
        // as many waves as have a piece of the row, up to four (eight for rows of 8 KiB: 1000 tokens of 2 rows 11.3 us
        // for 8.6, 8192 86 for 64)
        if (items <= 64)
            return far ? launch(moe_unpermute_backward_kernel<true, B, 1>, 1, item)
                       : launch(moe_unpermute_backward_kernel<false, B, 1>, 1, item);
        if (items <= 128)
            return far ? launch(moe_unpermute_backward_kernel<true, B, 2>, 2, item)
                       : launch(moe_unpermute_backward_kernel<false, B, 2>, 2, item);
        return far ? launch(moe_unpermute_backward_kernel<true, B, 4>, 4, item)
                   : launch(moe_unpermute_backward_kernel<false, B, 4>, 4, item);
    };
    typedef Elem<true>::v8 b8;
    return bf16 ? pick(std::true_type{}, b8{}) : pick(std::false_type{}, h8{});
}

}  // namespace lowbit
