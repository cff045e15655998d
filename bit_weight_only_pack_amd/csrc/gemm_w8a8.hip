// gemm_w8a8.hip -- products of int8 codes with int8 codes on the int8 matrix
// cores, one fp32 scale per token row and one per output channel: dense
// (lowbit_gemm_w8a8) and for rows sorted by expert (lowbit_moe_gemm_w8a8).
//
//   y[m][n] = RNE( xs[m] * ws[n] * S[m][n] + bias[n] ),  S[m][n] = sum_k xq[m][k] * wq[n][k]
//
// S is an exact int32 for every K the entry points accept (|xq wq| <= 2^14, so
// K < 2^17), whatever the order of summation: splitting K over waves or
// workgroups changes no bit of the result.  The scales and the bias are applied
// in fp32, fl(fl(fl(S) * xs) * ws + bias) (`scaled` below, the one place that
// does it), S first so that two small scales cannot underflow before S has
// lifted them; the one rounding to the output type is the last.
//
// Both operands are row-major with K contiguous, which is the operand order of
// v_mfma_i32_16x16x64_i8 (lane l: row l % 16, K bytes 16 (l / 16) .. + 15), so
// weights need no re-packing.  The weight is the A operand and the activation
// the B operand: a lane then holds four consecutive channels of one token.
#include <algorithm>
#include <type_traits>

#include "w8a8_sort.hpp"

namespace lowbit {

namespace {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));

// The product and the bias in one rounding, and said so: left to the compiler's contraction, kernels could differ in it.
// Without a bias the sum is with zero, which rounds the product alone.
__device__ __forceinline__ float scaled(int s, float xs, float ws, float bias)
{
    return __builtin_fmaf((float)s * xs, ws, bias);
}

__device__ __forceinline__ void put(void *y, int64_t o, float v, int bf16)
{
    if (bf16)
        static_cast<__bf16 *>(y)[o] = (__bf16)v;
    else
        static_cast<_Float16 *>(y)[o] = (_Float16)v;
}

// Vectors of outputs and partial sums start at any element: rows of odd lengths
// are stored 16 bytes at a time too (global memory takes them at any address).
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef b8 b8_any __attribute__((aligned(2)));
typedef h8 h8_any __attribute__((aligned(2)));
typedef i4 i4_any __attribute__((aligned(4)));

// outputs o .. o + 7, the first `valid` of them
__device__ __forceinline__ void put8(void *y, int64_t o, const float *v, int valid, int bf16)
{
    if (valid < 8) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < valid) put(y, o + i, v[i], bf16);
    } else if (bf16) {
        b8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
        *reinterpret_cast<b8_any *>(static_cast<__bf16 *>(y) + o) = r;
    } else {
        h8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = (_Float16)v[i];
        *reinterpret_cast<h8_any *>(static_cast<_Float16 *>(y) + o) = r;
    }
}

// 16 bytes of a row at K offset k; bytes past K (a multiple of 8, at least 8) are zeros.  No branch: many of
// these are under way together.
__device__ __forceinline__ i4 row16(const int8_t *row, int k, int K)
{
    const i2 lo = *reinterpret_cast<const i2 *>(row + min(k, K - 8)), hi = *reinterpret_cast<const i2 *>(row + min(k + 8, K - 8));
    const int lm = k < K ? -1 : 0, hm = k + 8 < K ? -1 : 0;
    return i4{lo.x & lm, lo.y & lm, hi.x & hm, hi.y & hm};
}

// sum of the lanes' values up to and including the lane's, in registers (shuffles go through LDS)
__device__ __forceinline__ int wave_prefix_sum(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1, :2, :4, :8 within 16 lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
    return v;
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rs, uint32_t lane_off, int k, uint8_t *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)lds, 16, lane_off, k, 0, 0);
}

// s_waitcnt vmcnt(N), other counters untouched
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// ---------------------------------------------------------------- streaming
// Few rows: the weights' stream is the cost.  A workgroup takes CH channels and
// up to 8 XL rows; its WV waves share K out in units of 128 bytes (wave w has
// units WV u + w, so the waves together read whole spans of each row).  Every
// wave runs a ring of its own in LDS: LDS-direct loads bring a unit of the rows
// and of the channels NST units ahead, and the wave that loaded it is the one
// that reads it, so it waits for its own load counter and there is no barrier.
// Reading the next units through LDS instead of registers keeps 1 KB of each
// load in one piece and leaves the registers to the sums.  The int32 sums of the
// waves are added through LDS at the end.  Rows past the last, of the activation
// or the weight, are read as copies of the last one and not stored.
//
// Bound: the weights' bytes once (and some 2 us of start and end).  Measured
// (us, weights not in the caches), CH / WV / NST by column, and tiles of 64:
//                          16/8/3   32/8/2   64/4/2   tiles
//   1024 x 4096   1 row      2.8      3.7      4.6      8.1
//   4096 x 4096   1 row      4.5      4.9      5.7      9.1
//                16 rows     4.8      5.2      6.3      9.6
//                32 rows     5.6      6.1      7.9      8.5
//                64 rows     7.2*     8.0*    10.8      9.3     (* 16/8/2, 32/4/2)
//   6144 x 4096  16 rows     7.6      6.4      6.8      8.5
//                64 rows    11.5*     8.9*    11.2      9.5
//  14336 x 4096  16 rows    15.1     12.5     10.6     12.2
//                32 rows    16.9     13.8     11.9     12.4
//  28672 x 4096  16 rows    30.5     27.6     23.6     26.9     (117 MB: 5.0 TB/s)
//                32 rows    36.3     31.6     28.8     27.5
template <int CH, int WV, int NST, int XL>
constexpr int kRingBytes = WV * NST * (8 * XL + CH) * 128;

// rows `first` .. `last` - 1 of the output, at most 8 XL of them, channels n0 ..
template <int CH, int WV, int NST, int XL>
__device__ __forceinline__ void w8a8_stream_rows(const W8Args &p, uint8_t *ring, const int8_t *wb, const float *ws,
                                                 int first, int last, int n0)
{
    constexpr int NB = CH / 16, TB = XL > 1 ? XL / 2 : 1;      // blocks of 16 channels, of 16 tokens
    constexpr int L = XL + CH / 8, STAGE = (8 * XL + CH) * 128;   // loads of a unit, its bytes
    constexpr int THREADS = WV * 64, SUMS = (16 * TB * CH + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const int n_valid = min(CH, p.N - n0), m_valid = last - first;
    const int units = p.K / 128;                      // whole ones
    const int mine = units > wave ? (units - wave + WV - 1) / WV : 0;

    // what the sums that this thread finishes are multiplied with
    const int n = tid % CH;
    const float wscale = ws[min(n, n_valid - 1)], bias = p.bias ? p.bias[n0 + min(n, n_valid - 1)] : 0.f;
    float xs[SUMS];
#pragma unroll
    for (int j = 0; j < SUMS; ++j)
        xs[j] = p.xs[w8a8_source_row(p, first + min((j * THREADS + tid) / CH, m_valid - 1))];
    // K behind the whole units: 64 bytes of the first waves
    const int k0 = units * 128 + wave * 64;
    i4 xt[TB], wt[NB];
    if (k0 < p.K) {
#pragma unroll
        for (int b = 0; b < TB; ++b)
            xt[b] = row16(p.x + (int64_t)w8a8_source_row(p, first + min(b * 16 + r16, m_valid - 1)) * p.K, k0 + kq * 16, p.K);
#pragma unroll
        for (int b = 0; b < NB; ++b)
            wt[b] = row16(wb + (int64_t)min(b * 16 + r16, n_valid - 1) * p.K, k0 + kq * 16, p.K);
    }

    // a load fills 8 rows of 128 bytes; chunk c of row r lies at c ^ (r / 2 % 8), so that the 16 rows which LDS
    // serves together lie in different banks
    const auto wrs = buffer_rsrc(wb, (uint32_t)((int64_t)n_valid * p.K));
    const int8_t *xp[XL];
    uint32_t off[CH / 8];
    const int put_chunk = ((lane & 7) ^ (lane >> 4)) * 16;
#pragma unroll
    for (int i = 0; i < XL; ++i)
        xp[i] = p.x + (int64_t)w8a8_source_row(p, first + min(8 * i + (lane >> 3), m_valid - 1)) * p.K +
                (put_chunk ^ (i & 1) * 64);
#pragma unroll
    for (int i = 0; i < CH / 8; ++i)
        off[i] = (uint32_t)min(8 * i + (lane >> 3), n_valid - 1) * (uint32_t)p.K + (put_chunk ^ (i & 1) * 64);
    uint8_t *own = ring + wave * NST * STAGE;
    auto issue = [&](int u, int slot) __attribute__((always_inline)) {
        const int k = (u * WV + wave) * 128;
        uint8_t *to = own + slot * STAGE;
#pragma unroll
        for (int i = 0; i < XL; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xp[i] + k),
                                             (__attribute__((address_space(3))) void *)(to + i * 1024), 16, 0, 0);
#pragma unroll
        for (int i = 0; i < CH / 8; ++i) dma16(wrs, off[i], k, to + (XL + i) * 1024);
    };
    i4 acc[TB][NB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[t][b] = i4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < NST; ++u)
        if (u < mine) issue(u, u);

    int slot = 0;
    for (int u = 0; u < mine; ++u) {
        // unit u has landed: where NST - 1 more are under way their loads may stay so, else all are waited for
        __builtin_amdgcn_sched_barrier(0);
        if (u + NST <= mine)
            wait_vm<(NST - 1) * L>();
        else
            wait_vm<0>();
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t *st = own + slot * STAGE;
        i4 x[TB][2], w[NB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = ((4 * h + kq) ^ (r16 >> 1)) * 16;
#pragma unroll
            for (int t = 0; t < TB; ++t)
                x[t][h] = XL == 1 ? *reinterpret_cast<const i4 *>(st + (r16 & 7) * 128 + ((4 * h + kq) ^ ((r16 & 7) >> 1)) * 16)
                                  : *reinterpret_cast<const i4 *>(st + (t * 16 + r16) * 128 + at);
#pragma unroll
            for (int b = 0; b < NB; ++b)
                w[b][h] = *reinterpret_cast<const i4 *>(st + XL * 1024 + (b * 16 + r16) * 128 + at);
        }
        // in registers: the slot is free
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (u + NST < mine) issue(u + NST, slot);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[t][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[b][h], x[t][h], acc[t][b], 0, 0, 0);
        slot = slot + 1 == NST ? 0 : slot + 1;
    }
    if (k0 < p.K)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                acc[t][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wt[b], xt[t], acc[t][b], 0, 0, 0);

    __syncthreads();                                  // every ring is done with
    int *part = reinterpret_cast<int *>(ring);        // [waves][16 TB][CH]
    static_assert(THREADS % CH == 0, "a thread finishes sums of one channel");
    static_assert(WV * 16 * TB * CH * 4 <= kRingBytes<CH, WV, NST, XL>, "the sums fit the rings");
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)                  // lane: token r16, channels 4 kq .. 4 kq + 3
            *reinterpret_cast<i4 *>(part + ((wave * TB + t) * 16 + r16) * CH + b * 16 + kq * 4) = acc[t][b];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SUMS; ++j) {
        const int i = j * THREADS + tid, m = i / CH;
        if (m >= m_valid || n >= n_valid) continue;
        int s = 0;
#pragma unroll
        for (int q = 0; q < WV; ++q) s += part[q * 16 * TB * CH + i];
        put(p.y, (int64_t)(first + m) * p.N + n0 + n, scaled(s, xs[j], wscale, bias), p.y_bf16);
    }
}

template <int CH, int WV, int NST, int XL>
__global__ __launch_bounds__(WV * 64) void w8a8_stream_kernel(W8Args p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[kRingBytes<CH, WV, NST, XL>];
    const int n0 = blockIdx.x * CH;
    w8a8_stream_rows<CH, WV, NST, XL>(p, ring, p.w + (int64_t)n0 * p.K, p.ws + n0, 0, p.rows, n0);
}

// By expert.  Row y < E of the grid is expert y's first 16 rows (or eight, where
// there are no more); the rows behind them, where an expert has more, are cut
// into runs of 16 that the remaining rows of the grid share.  They search the
// runs; the others, whose rows are most or all there are, start at once (128
// rows that reach some 65 of 128 experts of 1536 x 2048: 39 us; when this was
// chosen 45, and 57 with the search in all).
template <int CH, int WV, int NST>
__global__ __launch_bounds__(WV * 64) void w8a8_stream_experts_kernel(W8Args p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[kRingBytes<CH, WV, NST, 2>];
    const int n0 = blockIdx.x * CH, lane = threadIdx.x & 63;
    auto at = [&](int e) __attribute__((always_inline)) { return min(max(p.offsets[min(e, p.E)], 0), p.rows); };
    auto run = [&](int e, int first, int last) __attribute__((always_inline)) {
        const int64_t row = (int64_t)e * p.N + n0;
        if (last - first > 8)
            w8a8_stream_rows<CH, WV, NST, 2>(p, ring, p.w + row * p.K, p.ws + row, first, min(first + 16, last), n0);
        else
            w8a8_stream_rows<CH, WV, NST, 1>(p, ring, p.w + row * p.K, p.ws + row, first, last, n0);
    };
    int e = blockIdx.y, first, last, next = e - p.E;
    if (next < 0) {
        first = at(e);
        last = at(e + 1);
        if (first < last) run(e, first, last);
        return;
    }
    for (;; next += gridDim.y - p.E) {
        // run `next`: 64 experts at a time, one a lane
        int in = next;
        bool found = false;
        for (int e0 = 0; e0 < p.E && !found; e0 += 64) {
            const int low = at(e0 + lane), high = at(e0 + lane + 1), mine = max((high - low + 15) / 16 - 1, 0);
            const int incl = wave_prefix_sum(mine);
            const int all = __builtin_amdgcn_readlane(incl, 63);
            if (in < all) {
                const int l = __ffsll((unsigned long long)__ballot(incl > in)) - 1;
                e = e0 + l;
                first = __builtin_amdgcn_readlane(low, l) + 16 * (in - __builtin_amdgcn_readlane(incl - mine, l) + 1);
                last = __builtin_amdgcn_readlane(high, l);
                found = true;
            }
            in -= all;
        }
        if (!found) return;
        run(e, first, last);
        __syncthreads();                              // the sums are read before the next rows' rings are filled
    }
}

// ---------------------------------------------------------------- tiles
// One workgroup per BM tokens x BN channels, K in steps of BK bytes.  Both tiles
// move to LDS with LDS-direct 16-byte loads into a ring of NST stages, and from
// there to registers one K step ahead of the matrix instructions that use them.
// Rows of a stage are BK bytes; the 16-byte chunk c of row r lies at c ^ (r /
// SAME % C16), so that the 16 rows which LDS serves together lie in different
// banks.
//
// What bounds them, with the figures measured:
//   256 x 256  the matrix cores: 4096 x 4096 of K = 14336 in 195 to 204 us (2.4 to
//              2.5e15 operations/s), 171 with no load and no LDS read left in the
//              loop.  Per byte brought to LDS it does twice the work of 128 x 128;
//              one wave a SIMD, so a start and an end (14 us) that nothing hides.
//   128 x 256  bytes from L2 to LDS, three quarters of those of 128 x 128; three
//              stages, two waves a SIMD: 32768 rows with 128 experts of 1536 x 2048
//              in 201 us (codes of the whole range; 204 in tiles of 128 x 128, 216
//              in tiles of 256 x 256).
//   128 x 128  bytes from L2 to LDS: the same product moves 2.4 GB in its 204 us,
//              the matrix cores busy 28 % of the time, bytes from memory 1.09 times
//              the least.  Two workgroups a CU hide each other's starts and ends,
//              which counts where K is short (2048 x 768: 82 us, 88 in 128 x 256).
//   64 x 64    latency: few tiles (77 x 5003 of K = 4104: 10.5 us, 158 of them), so
//              all waves share one tile's K, and four stages are under way.
typedef int i16v __attribute__((ext_vector_type(16)));

// The tile of this workgroup among the tiles of all experts (their rows cut
// into runs of BM): consecutive numbers go over an expert's row tiles first, so
// that they share its weights.  False if there are fewer tiles, and for offsets
// that overlap (row ranges of a table that does not ascend).
struct W8Tile {
    int e, first, last, n0;
};

// P: experts a lane has, one after the other, at most.  Their offsets are loaded
// together and stay in registers: one wait for memory (1.0 us of the 21 that a
// tile of 128 x 128 with K = 2048 takes; 2.1 with a second look at the offsets
// and shuffles for the sum).
template <int BM, int BN, int P>
__device__ __forceinline__ bool expert_tile(const W8Args &p, W8Tile &t)
{
    const int lane = threadIdx.x & 63;
    const int nt = (p.N + BN - 1) / BN;
    const int per = (p.E + 63) / 64, e0 = lane * per;
    int at[P + 1];                                    // where the lane's experts begin, and its last one ends
#pragma unroll
    for (int i = 0; i <= P; ++i) at[i] = p.offsets[min(e0 + min(i, per), p.E)];
    int mine = 0;
#pragma unroll
    for (int i = 0; i <= P; ++i) {
        at[i] = min(max(at[i], 0), p.rows);
        if (i > 0) mine += (max(at[i] - at[i - 1], 0) + BM - 1) / BM;
    }
    const int incl = wave_prefix_sum(mine);
    // More than offsets that ascend can give: a damaged table, whose tiles times nt might pass 32 bits.  Up to here
    // they are no more than were launched.
    const int all = __builtin_amdgcn_readlane(incl, 63);
    if (all > p.rows / BM + p.E) return false;
    const int total = all * nt;
    const int run = (total + 7) / 8;                  // each XCD takes a run of tiles
    const int slot = blockIdx.x >> 3, lin = (blockIdx.x & 7) * run + slot;
    if (slot >= run || lin >= total) return false;
    // the lane whose experts have it, then the expert among them
    const int l = __ffsll((unsigned long long)__ballot(incl * nt > lin)) - 1;
    int in = lin - __builtin_amdgcn_readlane(incl - mine, l) * nt, low = 0, high = 0, tiles = 1;
    bool found = false;
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (!found) {
            low = __builtin_amdgcn_readlane(at[i], l);
            high = __builtin_amdgcn_readlane(at[i + 1], l);
            tiles = (max(high - low, 0) + BM - 1) / BM;
            t.e = l * per + i;
            found = in < tiles * nt;
            if (!found) in -= tiles * nt;
        }
    t.first = low + in % tiles * BM;
    t.last = high;
    t.n0 = in / tiles * BN;
    return true;
}

// DENSE, SPLIT: K over workgroups, int32 partial sums out; EXPERTS: rows by expert
enum W8Mode { DENSE, SPLIT, EXPERTS };

// What a tile's workgroup keeps in LDS
template <int BM, int BN, int NW, int BK, int NST>
struct W8Shared {
    static constexpr int NS = (BM + 2 * BN + NW * 64 - 1) / (NW * 64);
    __attribute__((aligned(1024))) uint8_t stages[NST * (BM + BN) * BK];
    __attribute__((aligned(16))) float sc[NS * NW * 64];      // token scales, channel scales, biases
};

// tile t, K steps s0 .. s1 - 1 of BK bytes
template <int BM, int BN, int NW, int BK, int NST, W8Mode MODE>
__device__ __forceinline__ void w8a8_tile(const W8Args &p, const W8Tile t, const int s0, const int s1, const int split,
                                          uint8_t *stages, float *sc)
{
    // 64 x 64: each wave has the whole tile and 32 bytes of every stage's K, so that no operand is read from LDS
    // twice; otherwise the waves share its area.
    constexpr bool KW = BM * BN == 64 * 64;
    static_assert(!KW || BK == 32 * NW, "a wave has 32 bytes of K");
    constexpr int NK = KW ? 1 : BK / 32;              // 32-byte pieces of a step that a wave multiplies
    constexpr int WC = KW ? 1 : NW / 2;               // waves side by side along the channels; two along the tokens
    constexpr int TC = BN / 32 / WC, TT = KW ? 2 : BM / 64;   // 32-wide blocks of a wave: channels, tokens
    constexpr int C16 = BK / 16, RPL = 64 / C16;      // 16-byte chunks of a row, rows of one LDS-direct load
    constexpr int LX = BM / RPL / NW, LW = BN / RPL / NW;   // such loads of a wave per stage
    constexpr int STAGE = (BM + BN) * BK;
    constexpr int SAME = 256 / BK;                    // rows in 256 bytes: all of LDS's banks
    static_assert(RPL * NW / SAME % C16 == 0, "every load stores its chunks in the same order");
    constexpr int THREADS = NW * 64, NS = W8Shared<BM, BN, NW, BK, NST>::NS;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wt = KW ? 0 : wave & 1, wc = KW ? 0 : wave >> 1;
    const int full = p.K / BK;
    const int m_valid = min(BM, t.last - t.first), n_valid = min(BN, p.N - t.n0);
    const int8_t *xb = MODE == EXPERTS && p.row_slot ? p.x : p.x + (int64_t)t.first * p.K;
    const int8_t *wb = p.w + ((int64_t)t.e * p.N + t.n0) * p.K;

    const int64_t x_bytes = (int64_t)(MODE == EXPERTS && p.row_slot ? p.x_rows : m_valid) * p.K;
    const auto xrs = buffer_rsrc(xb, (uint32_t)min(x_bytes, (int64_t)UINT32_MAX));
    const auto wrs = buffer_rsrc(wb, (uint32_t)((int64_t)n_valid * p.K));

    // load i of the wave fills LDS rows RPL (NW i + wave) .. + RPL - 1, lane -> (row, stored chunk)
    const int chunk0 = (lane & (C16 - 1)) ^ ((RPL * wave + lane / C16) / SAME & (C16 - 1));
    auto place = [&](uint8_t *buf, int i) __attribute__((always_inline)) {
        return buf + (i < LX ? 0 : BM * BK) + (NW * (i < LX ? i : i - LX) + wave) * 1024;
    };
    uint32_t off[LX + LW];
#pragma unroll
    for (int i = 0; i < LX + LW; ++i) {
        const int row = RPL * (NW * (i < LX ? i : i - LX) + wave) + lane / C16;
        int src = min(row, (i < LX ? m_valid : n_valid) - 1);
        if (MODE == EXPERTS && i < LX && p.row_slot) src = w8a8_source_row(p, t.first + src);
        off[i] = (uint32_t)src * (uint32_t)p.K + chunk0 * 16;
    }
    // the scales and biases of the tile, on their way while K is walked; every lane loads, so that no
    // branch makes the compiler wait
    float scale[NS];
    if constexpr (MODE != SPLIT)
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int i = j * THREADS + tid, r = t.first + min(i, m_valid - 1);
            const int n = t.n0 + min((i - BM) & (BN - 1), n_valid - 1);
            const float *from = p.xs + (MODE == EXPERTS ? w8a8_source_row(p, r) : r);
            if (i >= BM) from = p.ws + (int64_t)t.e * p.N + n;
            const bool none = i >= BM + BN && p.bias == nullptr;
            if (i >= BM + BN && !none) from = p.bias + n;
            const float v = *from;
            scale[j] = none ? 0.f : v;
        }

    auto load_one = [&](int s, uint8_t *buf, int i) __attribute__((always_inline)) {
        dma16(i < LX ? xrs : wrs, off[i], s * BK, place(buf, i));
    };
    // KW: K behind the last whole step, each wave 32 bytes of it straight to registers and multiplied while the first
    // stages are under way (77 x 5003 of K = 4104: 10.5 us, 11.7 as one more step through LDS)
    const int k_tail = full * BK + wave * 32;
    const bool tail = KW && k_tail < p.K && (MODE != SPLIT || split == p.splits - 1);
    i4 wl[TC], xl[TT];
    if (tail) {
#pragma unroll
        for (int c = 0; c < TC; ++c)
            wl[c] = row16(wb + (int64_t)min(c * 32 + (lane & 31), n_valid - 1) * p.K, k_tail + (lane >> 5) * 16, p.K);
#pragma unroll
        for (int b = 0; b < TT; ++b) {
            int src = min(b * 32 + (lane & 31), m_valid - 1);
            if (MODE == EXPERTS && p.row_slot) src = w8a8_source_row(p, t.first + src);
            xl[b] = row16(xb + (int64_t)src * p.K, k_tail + (lane >> 5) * 16, p.K);
        }
    }
    // the step that K ends inside, or an empty one that makes up a pair: bytes past K are zeros
    auto load_tail = [&](int s, uint8_t *buf) __attribute__((always_inline)) {
        const int k = s * BK + chunk0 * 16;
        constexpr int G = (LX + LW) % 4 == 0 ? 4 : (LX + LW) % 2 == 0 ? 2 : 1;
#pragma unroll
        for (int j = 0; j < LX + LW; j += G) {
            i4 v[G];
#pragma unroll
            for (int i = 0; i < G; ++i)
                v[i] = !KW && s * BK < p.K ? row16((j + i < LX ? xb : wb) + (off[j + i] - chunk0 * 16), k, p.K)
                                        : i4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < G; ++i) *reinterpret_cast<i4 *>(place(buf, j + i) + lane * 16) = v[i];
        }
    };
    auto load_stage = [&](int s, uint8_t *buf) __attribute__((always_inline)) {
        if (s < full) {
#pragma unroll
            for (int i = 0; i < LX + LW; ++i) load_one(s, buf, i);
        } else {
            load_tail(s, buf);
        }
    };
    // This wave's LDS reads are done, and its loads, but for those of the last `under_way` stages; then
    // everybody's.
    auto sync = [&](auto under_way) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        wait_vm<decltype(under_way)::value * (LX + LW)>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // operand addresses: row lane % 32 of a block, K chunk 2 k + lane / 32
    int at[NK];
#pragma unroll
    for (int k = 0; k < NK; ++k)
        at[k] = (lane & 31) * BK + ((2 * (KW ? wave : k) + (lane >> 5)) ^ ((lane & 31) / SAME & (C16 - 1))) * 16;
    auto token = [&](const uint8_t *buf, int b, int k) __attribute__((always_inline)) {
        return *reinterpret_cast<const i4 *>(buf + (wt * TT + b) * 32 * BK + at[k]);
    };
    auto channel = [&](const uint8_t *buf, int b, int k) __attribute__((always_inline)) {
        return *reinterpret_cast<const i4 *>(buf + BM * BK + (wc * TC + b) * 32 * BK + at[k]);
    };

    i16v acc[TC][TT];
#pragma unroll
    for (int c = 0; c < TC; ++c)
#pragma unroll
        for (int b = 0; b < TT; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c][b][i] = 0;

    // Where the accumulators leave room for two sets of operands, the next
    // step's are all read while this step's are used.
    constexpr bool kRoom = TC * TT < 16;
    constexpr int P2 = kRoom ? 2 : 1;
    // stage s is loaded by LDS-direct loads up to `direct`, then through registers
    const int direct = min(s1, full);
#pragma unroll
    for (int i = 0; i < NST; ++i)
        if (i < 2 ? s0 < s1 : s0 + i < s1) load_stage(s0 + i, stages + i * STAGE);
    if (tail)
#pragma unroll
        for (int c = 0; c < TC; ++c)
#pragma unroll
            for (int b = 0; b < TT; ++b)
                acc[c][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wl[c], xl[b], acc[c][b], 0, 0, 0);
    if (s0 < s1) {
        if (s0 + NST <= direct)
            sync(std::integral_constant<int, NST - 1>{});
        else
            sync(std::integral_constant<int, 0>{});
        uint8_t *const buf0 = stages;
        i4 wf[2][TC][NK], xf[P2][kRoom ? TT : 3][NK];
#pragma unroll
        for (int k = 0; k < NK; ++k) {
#pragma unroll
            for (int c = 0; c < TC; ++c) wf[0][c][k] = channel(buf0, c, k);
#pragma unroll
            for (int b = 0; b < (kRoom ? TT : 1); ++b) xf[0][b][k] = token(buf0, b, k);
        }
        auto step = [&](int s, uint8_t *cur, uint8_t *nxt, auto par) __attribute__((always_inline)) {
            constexpr int P = decltype(par)::value, Q = P ^ 1;
            const bool dma = s + NST < direct;
            // stage s is in registers everywhere, stage s + 1 in LDS
            auto next_stage = [&]() __attribute__((always_inline)) {
                if (NST > 2 && s + NST <= direct)
                    sync(std::integral_constant<int, NST - 2>{});
                else
                    sync(std::integral_constant<int, 0>{});
            };
            if constexpr (kRoom) {
                next_stage();
#pragma unroll
                for (int b = 0; b < TT; ++b)
#pragma unroll
                    for (int c = 0; c < TC; ++c) {
                        // this block's share of the next step's operands and of the loads two steps ahead
#pragma unroll
                        for (int f = 0; f < (TC + TT) * NK; ++f)
                            if (f * TC * TT / ((TC + TT) * NK) == b * TC + c) {
                                const int fk = f / (TC + TT), fi = f % (TC + TT);
                                if (fi < TC)
                                    wf[Q][fi][fk] = channel(nxt, fi, fk);
                                else
                                    xf[Q][fi - TC][fk] = token(nxt, fi - TC, fk);
                            }
                        if (dma) {
#pragma unroll
                            for (int i = 0; i < LX + LW; ++i)
                                if (i * TC * TT / (LX + LW) == b * TC + c) load_one(s + NST, cur, i);
                        }
#pragma unroll
                        for (int k = 0; k < NK; ++k)
                            acc[c][b] =
                                __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[P][c][k], xf[P][b][k], acc[c][b], 0, 0, 0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            } else {
                // Four token blocks in three register sets: blocks 0 and 2 in set 0, 1 in set 1, 3 in set 2.
                // Blocks 1 to 3 are read while blocks 0 and 1 are used; behind the barrier everybody is done
                // with stage s, and the channels and block 0 of stage s + 1 follow.
                static_assert(kRoom || (TC == 4 && TT == 4), "the schedule is for 4 x 4 blocks");
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b == 2) next_stage();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (b == 0) xf[0][1][c] = token(cur, 1, c);
                        if (b == 1) {
                            xf[0][0][c] = token(cur, 2, c);
                            xf[0][2][c] = token(cur, 3, c);
                        }
                        if (b >= 2) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) wf[Q][2 * (b - 2) + h][c] = channel(nxt, 2 * (b - 2) + h, c);
                            if (b == 3) xf[0][0][c] = token(nxt, 0, c);
                            if (dma) {
#pragma unroll
                                for (int h = 0; h < (LX + LW) / 8; ++h)
                                    load_one(s + NST, cur, ((b - 2) * 4 + c) * ((LX + LW) / 8) + h);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[c][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
                                wf[P][c][k], xf[0][b == 3 ? 2 : b & 1][k], acc[c][b], 0, 0, 0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            if (s + NST < s1 && s + NST >= full) load_tail(s + NST, cur);
        };
        int at0 = 0;                                  // stage s's place
        for (int s = s0; s < s1; s += 2) {
            const int at1 = at0 + STAGE == NST * STAGE ? 0 : at0 + STAGE;
            const int at2 = at1 + STAGE == NST * STAGE ? 0 : at1 + STAGE;
            step(s, stages + at0, stages + at1, std::integral_constant<int, 0>{});
            step(s + 1, stages + at1, stages + at2, std::integral_constant<int, 1>{});
            at0 = at2;
        }
    }
    if constexpr (MODE != SPLIT)
#pragma unroll
        for (int j = 0; j < NS; ++j) sc[j * THREADS + tid] = scale[j];
    sync(std::integral_constant<int, 0>{});           // the stages are free, the scales are in LDS

    // A lane holds token lane % 32 of a block and channels 8 g + 4 (lane / 32) + 0 .. 3.  32 tokens at a
    // time go through LDS (16-byte chunk c of row r at c ^ r) and come back as rows, eight channels a lane,
    // in a loop: unrolled, this code is so long that fetching it takes longer than running it.
    constexpr int CW = BN / WC, CHUNKS = CW / 4;   // channels of a wave, their chunks in a row
    constexpr int REGION = 32 * CW * 4;
    static_assert(NW * REGION * (KW ? TT : 1) <= NST * STAGE, "the waves' rows fit");
    const int c8 = lane % (CW / 8) * 8, n = wc * CW + c8;
    f4 ws[2], bs[2];
    if constexpr (MODE != SPLIT)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ws[h] = *reinterpret_cast<const f4 *>(&sc[BM + n + 4 * h]);
            bs[h] = *reinterpret_cast<const f4 *>(&sc[BM + BN + n + 4 * h]);
        }
    auto stash = [&](int b, uint8_t *region) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < TC; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<i4 *>(region + (lane & 31) * (CW * 4) +
                                        (((c * 8 + 2 * g + (lane >> 5)) ^ (lane & (CHUNKS - 1))) * 16)) =
                    i4{acc[c][b][4 * g], acc[c][b][4 * g + 1], acc[c][b][4 * g + 2], acc[c][b][4 * g + 3]};
    };
    auto fetch = [&](const uint8_t *region, int r, int h) __attribute__((always_inline)) {
        return *reinterpret_cast<const i4 *>(region + r * (CW * 4) + (((c8 / 4 + h) ^ (r & (CHUNKS - 1))) * 16));
    };
    auto emit = [&](int tok, const i4 *v) __attribute__((always_inline)) {
        if (tok >= m_valid) return;
        const int64_t o = (int64_t)(t.first + tok) * p.N + t.n0 + n;
        if constexpr (MODE == SPLIT) {
            int32_t *to = p.part + (int64_t)split * p.rows * p.N + o;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (n + 4 * h + 4 <= n_valid) {
                    *reinterpret_cast<i4_any *>(to + 4 * h) = v[h];
                } else {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (n + 4 * h + i < n_valid) to[4 * h + i] = v[h][i];
                }
        } else {
            const float xs = sc[tok];
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = scaled(v[i / 4][i % 4], xs, ws[i / 4][i % 4], bs[i / 4][i % 4]);
            put8(p.y, o, f, n_valid - n, p.y_bf16);
        }
    };
    if constexpr (KW) {
        // every wave's sums of the tile; then eight lanes add up and finish a row
#pragma unroll
        for (int b = 0; b < TT; ++b) stash(b, stages + (wave * TT + b) * REGION);
        sync(std::integral_constant<int, 0>{});
#pragma unroll
        for (int row = tid / 8; row < BM; row += THREADS / 8) {
            i4 v[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int q = 0; q < NW; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h) v[h] += fetch(stages + (q * TT + row / 32) * REGION, row % 32, h);
            emit(row, v);
        }
    } else {
        uint8_t *mine = stages + wave * REGION;
        constexpr int RSTEP = 64 / (CW / 8);
#pragma unroll
        for (int b = 0; b < TT; ++b) {
            const int tok0 = (wt * TT + b) * 32;
            stash(b, mine);
#pragma unroll 4
            for (int r = lane / (CW / 8); r < 32; r += RSTEP) {
                const i4 v[2] = {fetch(mine, r, 0), fetch(mine, r, 1)};
                emit(tok0 + r, v);
            }
        }
    }
}

template <int BM, int BN, int NW, int BK, int NST, W8Mode MODE>
__global__ __launch_bounds__(NW * 64, 1)
void w8a8_tile_kernel(W8Args p)
{
    __shared__ W8Shared<BM, BN, NW, BK, NST> sh;
    W8Tile t;
    // K in steps of BK bytes, in pairs; tiles of 64 take its end on their own
    const int full = p.K / BK, steps = BM * BN == 64 * 64 || full * BK == p.K ? full : full + 1;
    int s0 = 0, s1 = (steps + 1) / 2 * 2, split = 0;
    if constexpr (MODE == EXPERTS) {
        if (!(p.E <= 256 ? expert_tile<BM, BN, 4>(p, t) : expert_tile<BM, BN, 16>(p, t))) return;
    } else {
        // each XCD takes a run of tiles, which covers blocks of 8 token tiles
        const uint32_t mt = (p.rows + BM - 1) / BM, nt = (p.N + BN - 1) / BN;
        const uint32_t tiles = mt * nt, all = MODE == SPLIT ? tiles * p.splits : tiles, per = (all + 7) / 8;
        const uint32_t slot = blockIdx.x >> 3, lin = (blockIdx.x & 7) * per + slot;
        if (slot >= per || lin >= all) return;
        uint32_t in = lin;
        if constexpr (MODE == SPLIT) {
            split = lin / tiles;
            in = lin % tiles;
            const int pairs = s1 / 2;
            s0 = (int)((int64_t)pairs * split / p.splits) * 2;
            s1 = (int)((int64_t)pairs * (split + 1) / p.splits) * 2;
        }
        const uint32_t group = in / (8 * nt);
        const uint32_t high = min(8u, mt - group * 8), rest = in - group * 8 * nt;
        t.e = 0;
        t.first = (group * 8 + rest % high) * BM;
        t.last = p.rows;
        t.n0 = rest / high * BN;
    }
    // An expert's last tile with half its rows or fewer is done as half a tile: it moves fewer bytes and multiplies half
    // as much (128 experts of 1536 x 2048, us: 128 rows each 133 in tiles of 128 and 129 in tiles of 256, 143 and 142
    // without; 256 rows 217 and 235, 221 and 249).
    if constexpr (MODE == EXPERTS && BM > 64)
        if (t.last - t.first <= BM / 2) {
            w8a8_tile<BM / 2, BN, NW, BK, NST, MODE>(p, t, s0, s1, split, sh.stages, sh.sc);
            return;
        }
    w8a8_tile<BM, BN, NW, BK, NST, MODE>(p, t, s0, s1, split, sh.stages, sh.sc);
}

// Sums of the splits' planes, in their order, scaled and rounded: four channels of a row a thread
__global__ __launch_bounds__(256) void w8a8_reduce_kernel(W8Args p)
{
    const int64_t MN = (int64_t)p.rows * p.N, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int groups = (p.N + 3) / 4;
    if (i >= (int64_t)p.rows * groups) return;
    const int m = (int)(i / groups), n = (int)(i - (int64_t)m * groups) * 4;
    const int64_t o = (int64_t)m * p.N + n;
    const float xs = p.xs[m];
    if (n + 4 <= p.N) {
        i4 s = *reinterpret_cast<const i4_any *>(p.part + o);
        for (int q = 1; q < p.splits; ++q) s += *reinterpret_cast<const i4_any *>(p.part + q * MN + o);
        f4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = scaled(s[j], xs, p.ws[n + j], p.bias ? p.bias[n + j] : 0.f);
        if (p.y_bf16) {
            typedef __bf16 b4 __attribute__((ext_vector_type(4)));
            typedef b4 b4_any __attribute__((aligned(2)));
            *reinterpret_cast<b4_any *>(static_cast<__bf16 *>(p.y) + o) = __builtin_convertvector(v, b4);
        } else {
            typedef _Float16 h4 __attribute__((ext_vector_type(4)));
            typedef h4 h4_any __attribute__((aligned(2)));
            *reinterpret_cast<h4_any *>(static_cast<_Float16 *>(p.y) + o) = __builtin_convertvector(v, h4);
        }
        return;
    }
    for (int j = 0; n + j < p.N; ++j) {
        int s = p.part[o + j];
        for (int q = 1; q < p.splits; ++q) s += p.part[q * MN + o + j];
        put(p.y, o + j, scaled(s, xs, p.ws[n + j], p.bias ? p.bias[n + j] : 0.f), p.y_bf16);
    }
}

void reduce_launch(const W8Args &a, hipStream_t s)
{
    const int64_t threads = (int64_t)a.rows * ((a.N + 3) / 4);
    w8a8_reduce_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(a);
}

}  // namespace

namespace {

constexpr int kCUs = 256;

template <int CH, int WV, int NST, int XL>
void stream(const W8Args &a, hipStream_t s)
{
    w8a8_stream_kernel<CH, WV, NST, XL><<<(a.N + CH - 1) / CH, WV * 64, 0, s>>>(a);
}

// The kernel a product takes: streaming, or tiles of rows x channels with K
// split over `splits` workgroups.
struct W8Choice {
    bool stream;
    int rows, channels, waves;                        // of a workgroup
    int splits;
    int64_t tiles;                                    // workgroups of the tile kernel (by expert: at most)
};

// As few channels a workgroup as give every CU one, as many rows as there are.
W8Choice stream_choice(int rows, int N)
{
    const int up_to = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    if (N <= 16 * kCUs) return {true, up_to, 16, 8, 1, 0};
    if (up_to > 16 || N <= 32 * kCUs) return {true, up_to, 32, up_to == 64 ? 4 : 8, 1, 0};
    return {true, up_to, 64, 4, 1, 0};
}

template <int XL>
void stream(const W8Args &a, const W8Choice &c, hipStream_t s)
{
    constexpr bool kMany = XL == 8;                   // the rings of 64 rows leave room for less
    if (c.channels == 16)
        stream<16, 8, kMany ? 2 : 3, XL>(a, s);
    else if (XL > 2 || c.channels == 32)
        stream<32, kMany ? 4 : 8, 2, XL>(a, s);
    else if constexpr (XL <= 2)
        stream<64, 4, 2, XL>(a, s);
}

template <int CH, int WV, int NST>
void stream_experts(const W8Args &a, hipStream_t s)
{
    // for the runs behind the experts' first: eight, or one for every eight runs there may be (rows past the tile
    // kernel's reach can be many: a grid has fewer than 2^16 rows)
    const int more = min(a.rows / 16, max(8, min(a.rows / 128, 1 << 15)));
    w8a8_stream_experts_kernel<CH, WV, NST><<<dim3((a.N + CH - 1) / CH, a.E + more), WV * 64, 0, s>>>(a);
}

template <int BM, int BN, int NW, int BK, int NST, W8Mode MODE>
void tile_launch(const W8Args &a, int64_t tiles, hipStream_t s)
{
    w8a8_tile_kernel<BM, BN, NW, BK, NST, MODE><<<(unsigned)round_up(tiles, 8), NW * 64, 0, s>>>(a);
}

// Tiles of rows x channels and the estimated time (us) of a launch of them: a
// start and an end, then per 128 bytes of K a time for each tile a CU has to
// take and one for the tile's own start and end; or, where a CU has no more than
// one, a time for K alone.  The constants are fitted to the choice among 3100
// launches (195 shapes of 371 to 28672 channels, K 192 to 14336 and 69 to 4096
// rows, unsplit and split; 30 by expert): it takes 0.6 % longer than the best of
// them on average, 21 % at most.  Best of these kernels, that is: the operations
// or bytes alone would take a quarter to two thirds of it between 70 and 2200 rows.
struct W8Cost {
    int rows, channels;
    double ends, step, tile, alone;
};
constexpr W8Cost kCosts[] = {{64, 64, 3.85, 0.213, 0.51, 0.151},
                             {128, 128, 4.2, 0.516, 0.65, 0.769},
                             {128, 256, 5.57, 0.796, 2.63, 0.725},
                             {256, 256, 14.6, 1.286, 5.29, 1.102}};
constexpr int kSizes = sizeof(kCosts) / sizeof(kCosts[0]);

double tiles_time(const W8Cost &c, int64_t tiles, int pairs)
{
    const int64_t each = (tiles + kCUs - 1) / kCUs;
    return c.ends + (each > 1 ? each * (pairs * 2 * c.step + c.tile) : pairs * 2 * c.alone);
}

// Tiles of 64 x 64 share K among eight waves where a CU has no more than one of them.
W8Choice tile_choice(int size, int splits, int64_t tiles)
{
    const W8Cost &c = kCosts[size];
    const bool eight = c.rows == 64 ? tiles <= kCUs : c.rows != c.channels;
    return {false, c.rows, c.channels, eight ? 8 : 4, splits, tiles};
}

template <W8Mode MODE>
void tile_launch(const W8Args &a, const W8Choice &c, hipStream_t s)
{
    if (c.rows == 64 && c.waves == 8)
        tile_launch<64, 64, 8, 256, 4, MODE>(a, c.tiles, s);
    else if (c.rows == 64)
        tile_launch<64, 64, 4, 128, 4, MODE>(a, c.tiles, s);
    else if (c.channels == 128)
        tile_launch<128, 128, 4, 128, 2, MODE>(a, c.tiles, s);
    else if (c.rows == 128)
        tile_launch<128, 256, 8, 128, 3, MODE>(a, c.tiles, s);
    else
        tile_launch<256, 256, 4, 128, 2, MODE>(a, c.tiles, s);
}

struct W8Plan {
    int size, splits;                                 // of kCosts; workgroups that share K
    int64_t tiles;
    double time;
};

// One launch has that many tiles: a grid holds fewer than 2^32 threads.
bool grid_holds(const W8Cost &c, int64_t tiles)
{
    const int64_t threads = c.rows != c.channels ? 512 : 256;      // the tiles of 64 take 512 only where they are few
    return (int64_t)round_up(tiles, 8) * threads < (int64_t)1 << 32;
}

int64_t tiles_of(const W8Cost &c, int rows, int N)
{
    return (((int64_t)rows + c.rows - 1) / c.rows) * (((int64_t)N + c.channels - 1) / c.channels);
}

// The tile size and split with the least estimated time, of those that a grid
// holds.  A split adds the pass over the partial sums.
W8Plan w8_plan(int rows, int N, int K)
{
    const int pairs = (K + 255) / 256;
    W8Plan best = {0, 1, 0, -1.0};
    for (int i = 0; i < kSizes; ++i) {
        const W8Cost &c = kCosts[i];
        const int64_t tiles = tiles_of(c, rows, N);
        for (int splits = 1; splits <= 8 && (splits == 1 || splits * 2 <= pairs); splits *= 2) {
            if (!grid_holds(c, tiles * splits)) break;
            const double reduce = splits > 1 ? 3.5 + (double)splits * rows * N * 8 / 5.8e6 : 0.0;
            const double us = tiles_time(c, tiles * splits, (pairs + splits - 1) / splits) + reduce;
            if (best.time < 0.0 || us < best.time) best = {i, splits, tiles * splits, us};
        }
    }
    return best;
}

// A dense product streams the weights where one pass over them serves all rows
// faster than tiles do: up to 16 rows (16 rows, stream / tiles, us: 1024 channels
// of K = 14336 11.0 / 12.4, 4096 of 28672 25.0 / 26.8; tiles are ahead where few
// channels walk a very long K: 1024 of 28672 19.5 / 15.7, 64 of 131064 107 / 41;
// one row 12.8 / 14.8 and 62 / 33), and up to 64 by an estimate: a start and
// an end, then what a workgroup brings to its CU (faster where half of them have
// none) or the weights from memory.  Measured on 120 shapes of 24 to 64 rows, 200
// to 8192 channels, K 2048 to 28672, this takes 0.3 % longer than the better of
// both on average, 12 % at most (64 x 4096: K = 4096 7.2 us against 9.3 in tiles,
// K = 12432 19.7 against 15.8).
bool w8_streams(int rows, int N, int K)
{
    if (rows <= 16) return true;
    if (rows > 64 || N > 32 * kCUs) return false;
    const int channels = N <= 16 * kCUs ? 16 : 32, workgroups = (N + channels - 1) / channels;
    const double own = (double)K * (channels + (rows <= 32 ? 32 : 64)) / (workgroups > kCUs / 2 ? 72e3 : 90e3);
    return 2.0 + std::max(own, (double)N * K / 5e6) <= 1.1 * w8_plan(rows, N, K).time;
}

W8Choice dense_choice(int rows, int N, int K)
{
    if (w8_streams(rows, N, K)) return stream_choice(rows, N);
    const W8Plan pl = w8_plan(rows, N, K);
    return tile_choice(pl.size, pl.splits, pl.tiles);
}

}  // namespace

bool gemm_w8a8_fits(int M, int N)
{
    const W8Cost &most = kCosts[kSizes - 1];
    return M <= 16 || grid_holds(most, tiles_of(most, M, N));
}

size_t gemm_w8a8_workspace(int M, int N, int K)
{
    const W8Choice c = dense_choice(M, N, K);
    return c.splits > 1 ? (size_t)c.splits * M * N * sizeof(int32_t) : 0;
}

hipError_t launch_gemm_w8a8(const W8Args &args, void *ws, hipStream_t s)
{
    W8Args a = args;
    const W8Choice c = dense_choice(a.rows, a.N, a.K);
    if (c.stream) {
        if (c.rows == 8)
            stream<1>(a, c, s);
        else if (c.rows == 16)
            stream<2>(a, c, s);
        else if (c.rows == 32)
            stream<4>(a, c, s);
        else
            stream<8>(a, c, s);
        return hipGetLastError();
    }
    a.splits = c.splits;
    a.part = static_cast<int32_t *>(ws);
    if (c.splits > 1) {
        tile_launch<SPLIT>(a, c, s);
        reduce_launch(a, s);
    } else {
        tile_launch<DENSE>(a, c, s);
    }
    return hipGetLastError();
}

// Streaming goes by the rows that an expert has on average, tiles by their
// estimated time.  Measured (us, weights not in the caches), the same number of
// rows for every expert:
//   rows an expert                             1      4      8     12     16
//   128 experts of 1536 x 2048: stream        65     65     66     72     75     (403 MB: 6.2 TB/s with one row)
//                               tiles of 64   72     76     77     78     80
//   8 experts of 4096 x 4096:   stream        27     27     27     28     29
//                               tiles of 64   32     32     32     32     32
//   rows an expert                            64                       256
//   128 experts: tiles of 64 / 128 / 128 x 256 / 256
//                                             93 / 88 /  88 / 103     243 / 167 / 156 / 148
//   8 experts                                 34 / 40 /  39 /  53      76 /  53 /  49 /  68
// The estimate counts half a tile more for every expert: for 256 rows each, all
// tiles whole, it takes 128 x 256 for the 128 experts and 256 for the 8.  Routed
// rows, 128 experts of 1536 x 2048, stream / tiles of 64: 128 rows (66 experts
// reached) 36 / 43, 512 (107) 56 / 64, 1024 (121) 72 / 74, 1536 (122) 92 / 76; all
// 1536 rows with one of the experts: 46 / 16.
// A ring of four waves and three stages holds twelve units of K: with fewer of
// them two waves and two stages serve more workgroups a CU (128 experts of
// 2048 x 768, 1 / 4 / 8 rows each: 34 / 35 / 37 against 46 / 47 / 50; of
// 1536 x 2048: 66 / 68 / 69 against 65 / 65 / 66).
// Gathered rows of 4 GiB and more stream, however many: 64 / 512 / 4096 rows, 8
// experts of 4096 x 4096: 24 / 70 / 408 against 25 / 24 / 80 below 4 GiB.
// `rows` is what y holds, not the rows that exist: with 16 of 128 experts of
// 1536 x 2048 here and 64 / 256 / 1024 tokens of 8, 13 / 18 / 34 against 10 / 15
// / 16 with rows cut to those that exist.
//
// gathered: rows of x that row_slot picks from, 0 where rows lie in expert order
static W8Choice experts_choice(int E, int rows, int N, int K, int64_t gathered)
{
    // the rows' offsets inside x are 32-bit in the tile kernel when they are gathered
    const bool far = gathered * K >= (int64_t)1 << 32;
    const W8Choice few = {true, 16, 32, K < 12 * 128 ? 2 : 4, 1, 0};
    if (rows <= 12 * E || far) return few;
    // the size whose tiles take the least estimated time, an expert's last tile being half full and every expert
    // having a row; at most one more tile for each of them is launched.  Where no grid holds them (many experts of
    // millions of channels) the streaming kernel goes on: its runs of rows are shared by as many workgroups as there are
    int size = -1;
    int64_t most = 0;
    double time = 0.0;
    for (int i = 0; i < kSizes; ++i) {
        const W8Cost &c = kCosts[i];
        const int64_t nt = ((int64_t)N + c.channels - 1) / c.channels, whole = (int64_t)rows / c.rows;
        if (!grid_holds(c, (whole + E) * nt)) continue;
        const double us = tiles_time(c, std::max((int64_t)E, whole + E / 2) * nt, (K + 255) / 256);
        if (size < 0 || us < time) {
            size = i;
            most = (whole + E) * nt;
            time = us;
        }
    }
    return size < 0 ? few : tile_choice(size, 1, most);
}

hipError_t launch_moe_gemm_w8a8(const W8Args &a, hipStream_t s)
{
    const W8Choice c = experts_choice(a.E, a.rows, a.N, a.K, a.row_slot != nullptr ? a.x_rows : 0);
    if (!c.stream)
        tile_launch<EXPERTS>(a, c, s);
    else if (c.waves == 2)
        stream_experts<32, 2, 2>(a, s);
    else
        stream_experts<32, 4, 3>(a, s);
    return hipGetLastError();
}

}  // namespace lowbit

void lowbit_internal_w8a8_choice(int E, int rows, int N, int K, int gathered, int *choice)
{
    const lowbit::W8Choice c = E > 0 ? lowbit::experts_choice(E, rows, N, K, gathered) : lowbit::dense_choice(rows, N, K);
    const int of[] = {c.stream, c.rows, c.channels, c.waves, c.splits};
    std::copy(of, of + 5, choice);
}
