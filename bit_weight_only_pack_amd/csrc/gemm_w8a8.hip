// gemm_w8a8.hip -- products of int8 codes with int8 codes on the int8 matrix
// cores, one fp32 scale per token row and one per output channel: dense
// (lowbit_gemm_w8a8) and for rows sorted by expert (lowbit_moe_gemm_w8a8).
//
//   y[m][n] = RNE( xs[m] * ws[n] * S[m][n] + bias[n] ),  S[m][n] = sum_k xq[m][k] * wq[n][k]
//
// S is an exact int32 for every K the entry points accept (|xq wq| <= 2^14, so
// K < 2^17), whatever the order of summation: splitting K over waves or
// workgroups changes no bit of the result.  The scales are applied in fp32,
// fl(fl(S * xs) * ws), S first so that two small scales cannot underflow
// before S has lifted them; the one rounding to the output type is the last.
//
// Both operands are row-major with K contiguous, which is the operand order of
// v_mfma_i32_16x16x64_i8 (lane l: row l % 16, K bytes 16 (l / 16) .. + 15), so
// weights need no re-packing.  The weight is the A operand and the activation
// the B operand: a lane then holds four consecutive channels of one token.
#include <type_traits>

#include "w8a8_sort.hpp"

namespace lowbit {

namespace {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));
typedef int i4a __attribute__((ext_vector_type(4), aligned(8)));   // rows start at multiples of 8 bytes

__device__ __forceinline__ void put(void *y, int64_t o, float v, int bf16)
{
    if (bf16)
        static_cast<__bf16 *>(y)[o] = (__bf16)v;
    else
        static_cast<_Float16 *>(y)[o] = (_Float16)v;
}

__device__ __forceinline__ void put8(void *y, int64_t o, const float *v, int bf16)
{
    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
    if (bf16) {
        b8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
        *reinterpret_cast<b8 *>(static_cast<__bf16 *>(y) + o) = r;
    } else {
        h8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = (_Float16)v[i];
        *reinterpret_cast<h8 *>(static_cast<_Float16 *>(y) + o) = r;
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

// ---------------------------------------------------------------- streaming
// Few rows: the weights' stream is the cost.  A workgroup takes a run of 16
// channels for 16 rows at a time; its 8 waves share K out in units of 128 bytes
// (unit u of wave w is 8 u + w, so the waves together read whole spans of each
// row) and add their int32 sums through LDS.  Weights go straight to registers.
// Where U units are all of a wave's K, every load is under way at once; LOOP:
// the next U are loaded while U are multiplied.  Rows past the last (of the
// activation or the weight) are read as copies of the last one and not stored.
constexpr int W = 8;                                  // waves

template <int U, bool LOOP, bool GROUPED>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(4)))
void w8a8_stream_kernel(W8Args p)
{
    __shared__ __attribute__((aligned(16))) int part[W][256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const int n0 = blockIdx.x * 16;
    int first = 0, last = p.rows;
    const int8_t *w = p.w;
    const float *ws = p.ws;
    if constexpr (GROUPED) {
        const int e = blockIdx.y;
        first = max(p.offsets[e], 0);
        last = min(p.offsets[e + 1], p.rows);
        if (first >= last) return;
        w += (int64_t)e * p.N * p.K;
        ws += (int64_t)e * p.N;
    }
    w += (int64_t)n0 * p.K;
    const int units = p.K / 128;                      // whole ones
    const int mine = units > wave ? (units - wave + W - 1) / W : 0;
    const int nb = (mine + U - 1) / U;                // batches of this wave
    const uint32_t row = (uint32_t)min(r16, p.N - 1 - n0) * (uint32_t)p.K + kq * 16;
    const int tm = (tid >> 4) & 15, n = n0 + (tid & 15);   // the sum that this thread finishes
    const float wscale = ws[min(n, p.N - 1)];

    for (int m0 = first; m0 < last; m0 += 16) {
        const int8_t *xr = p.x + (int64_t)w8a8_source_row(p, min(m0 + r16, last - 1)) * p.K + kq * 16;
        const float xs = p.xs[w8a8_source_row(p, min(m0 + tm, last - 1))];
        i4 wv[LOOP ? 2 : 1][U][2], xv[LOOP ? 2 : 1][U][2], acc = {0, 0, 0, 0};
        auto load = [&](int b, i4 (&v)[U][2], i4 (&x)[U][2]) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!LOOP && u >= mine) continue;
                const int k = ((LOOP ? min(b * U + u, mine - 1) : u) * W + wave) * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[u][h] = __builtin_nontemporal_load(reinterpret_cast<const i4a *>(w + k + 64 * h + row));
                    x[u][h] = *reinterpret_cast<const i4a *>(xr + k + 64 * h);
                }
            }
        };
        auto multiply = [&](int b, const i4 (&v)[U][2], const i4 (&x)[U][2]) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (b * U + u < mine)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[u][h], x[u][h], acc, 0, 0, 0);
        };
        // K behind the whole units: 64 bytes of a wave
        const int k0 = units * 128 + wave * 64;
        i4 xt, wt;
        auto load_tail = [&]() __attribute__((always_inline)) {
            if (k0 >= p.K) return;
            xt = row16(xr - kq * 16, k0 + kq * 16, p.K);
            wt = row16(w + row - kq * 16, k0 + kq * 16, p.K);
        };
        if constexpr (!LOOP) {
            load(0, wv[0], xv[0]);
            load_tail();
            multiply(0, wv[0], xv[0]);
        } else if (nb > 0) {
            load(0, wv[0], xv[0]);
            int b = 0;
            for (; b + 2 < nb; b += 2) {
                load(b + 1, wv[1], xv[1]);
                multiply(b, wv[0], xv[0]);
                load(b + 2, wv[0], xv[0]);
                multiply(b + 1, wv[1], xv[1]);
            }
            if (b + 1 < nb) {
                load(b + 1, wv[1], xv[1]);
                multiply(b, wv[0], xv[0]);
                multiply(b + 1, wv[1], xv[1]);
            } else {
                multiply(b, wv[0], xv[0]);
            }
        }
        if (LOOP) load_tail();
        if (k0 < p.K) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wt, xt, acc, 0, 0, 0);
        // lane: token r16, channels 4 kq .. 4 kq + 3
        *reinterpret_cast<i4 *>(&part[wave][r16 * 16 + kq * 4]) = acc;
        __syncthreads();
        if (tid < 256) {
            int sum = 0;
#pragma unroll
            for (int q = 0; q < W; ++q) sum += part[q][tid];
            if (m0 + tm < last && n < p.N) {
                float v = (float)sum * xs * wscale;
                if (p.bias) v += p.bias[n];
                put(p.y, (int64_t)(m0 + tm) * p.N + n, v, p.y_bf16);
            }
        }
        if (m0 + 16 < last) __syncthreads();          // the sums are read before the next rows' are written
    }
}

// The same for many channels and several rows (dense): one workgroup per CU
// goes through runs of 16 channels, the rows' operands staying in registers
// and the next run's weights on their way while a run is finished.
template <int U>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(2)))
void w8a8_resident_kernel(W8Args p)
{
    __shared__ __attribute__((aligned(16))) int part[2][W][256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kq = lane >> 4;
    const int runs = (p.N + 15) / 16, step = gridDim.x;
    const int units = p.K / 128;
    const int mine = units > wave ? (units - wave + W - 1) / W : 0;
    const int tm = (tid >> 4) & 15, tn = tid & 15;    // the sum that this thread finishes
    const int8_t *xr = p.x + (int64_t)min(r16, p.rows - 1) * p.K + kq * 16;
    const float xs = p.xs[min(tm, p.rows - 1)];
    const int k0 = units * 128 + wave * 64;           // K behind the whole units: 64 bytes of a wave
    const i4 xt = k0 < p.K ? row16(xr - kq * 16, k0 + kq * 16, p.K) : i4{0, 0, 0, 0};
    i4 xv[U][2], wv[2][U][2], wt[2];
    float wscale[2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            xv[u][h] = *reinterpret_cast<const i4a *>(xr + (max(min(u, mine - 1), 0) * W + wave) * 128 + 64 * h);
    auto load = [&](int run, int to) __attribute__((always_inline)) {
        const int r = min(run, runs - 1);
        const int8_t *w = p.w + (int64_t)r * 16 * p.K;
        const uint32_t row = (uint32_t)min(r16, p.N - 1 - r * 16) * (uint32_t)p.K + kq * 16;
        wscale[to] = p.ws[min(r * 16 + tn, p.N - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wv[to][u][h] = __builtin_nontemporal_load(reinterpret_cast<const i4a *>(
                    w + (max(min(u, mine - 1), 0) * W + wave) * 128 + 64 * h + row));
        if (k0 < p.K) wt[to] = row16(w + row - kq * 16, k0 + kq * 16, p.K);
    };
    auto finish = [&](int run, int from) __attribute__((always_inline)) {
        i4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < mine)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[from][u][h], xv[u][h], acc, 0, 0, 0);
        if (k0 < p.K) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wt[from], xt, acc, 0, 0, 0);
        *reinterpret_cast<i4 *>(&part[from][wave][r16 * 16 + kq * 4]) = acc;
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // loads stay under way
        if (tid < 256) {
            int s = 0;
#pragma unroll
            for (int q = 0; q < W; ++q) s += part[from][q][tid];
            const int n = run * 16 + tn;
            if (tm < p.rows && n < p.N) {
                float v = (float)s * xs * wscale[from];
                if (p.bias) v += p.bias[n];
                put(p.y, (int64_t)tm * p.N + n, v, p.y_bf16);
            }
        }
        // the two halves of `part` take turns: a half is written again only behind the other's barrier,
        // which every wave passes after it has read the first
    };
    load(blockIdx.x, 0);
    for (int run = blockIdx.x; run < runs; run += 2 * step) {
        load(run + step, 1);
        finish(run, 0);
        if (run + step >= runs) break;
        load(run + 2 * step, 0);
        finish(run + step, 1);
    }
}

// ---------------------------------------------------------------- tiles
// One workgroup per BM tokens x BN channels, K in steps of BK bytes.  Both tiles
// move to LDS with LDS-direct 16-byte loads into a ring of NST stages, and from
// there to registers one K step ahead of the matrix instructions that use them.
// Rows of a stage are BK bytes; the 16-byte chunk c of row r lies at c ^ (r /
// SAME % C16), so that the 16 rows which LDS serves together lie in different
// banks.
typedef int i16v __attribute__((ext_vector_type(16)));

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

// The tile of this workgroup among the tiles of all experts (their rows cut
// into runs of BM): consecutive numbers go over an expert's row tiles first, so
// that they share its weights.  False if there are fewer tiles.
struct W8Tile {
    int e, first, last, n0;
};

template <int BM, int BN>
__device__ __forceinline__ bool expert_tile(const W8Args &p, W8Tile &t)
{
    const int lane = threadIdx.x & 63;
    const int nt = (p.N + BN - 1) / BN;
    // a lane has `per` experts one after the other; all their offsets are loaded at once
    const int per = (p.E + 63) / 64, e0 = lane * per;
    auto at = [&](int e) __attribute__((always_inline)) { return min(max(p.offsets[min(e, p.E)], 0), p.rows); };
    int mine = 0, low = at(e0);
    const int first = low;
#pragma unroll 4
    for (int i = 0; i < per; ++i) {
        const int high = at(e0 + i + 1);
        mine += (max(high - low, 0) + BM - 1) / BM;
        low = high;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63) * nt;
    const int run = (total + 7) / 8;                  // each XCD takes a run of tiles
    const int slot = blockIdx.x >> 3, lin = (blockIdx.x & 7) * run + slot;
    if (slot >= run || lin >= total) return false;
    // the lane whose experts have it, then the expert among them
    const int l = __ffsll((unsigned long long)__ballot(incl * nt > lin)) - 1;
    int in = lin - __builtin_amdgcn_readlane(incl - mine, l) * nt, e = l * per;
    low = __builtin_amdgcn_readlane(first, l);
    for (;; ++e) {
        const int high = at(e + 1), tiles = (max(high - low, 0) + BM - 1) / BM;
        if (in < tiles * nt) {
            t.e = e;
            t.first = low + in % tiles * BM;
            t.last = high;
            t.n0 = in / tiles * BN;
            return true;
        }
        in -= tiles * nt;
        low = high;
    }
}

// DENSE, SPLIT: K over workgroups, int32 partial sums out; EXPERTS: rows by expert
enum W8Mode { DENSE, SPLIT, EXPERTS };

template <int BM, int BN, int NW, W8Mode MODE>
__global__ __launch_bounds__(NW * 64, 1)
void w8a8_tile_kernel(W8Args p)
{
    constexpr int NST = BM * BN == 64 * 64 ? 4 : 2;   // LDS stages
    constexpr int BK = 32 * NW;                       // bytes of K in one
    // 64 x 64: each wave has the whole tile and 32 bytes of every stage's K, so that no operand is read from LDS
    // twice; otherwise each has a quarter of the tile.
    constexpr bool KW = BM * BN == 64 * 64;
    static_assert(KW || NW == 4, "2 x 2 waves share a tile");
    constexpr int NK = KW ? 1 : 4;                    // 32-byte pieces of a step that a wave multiplies
    constexpr int TC = KW ? 2 : BN / 64, TT = KW ? 2 : BM / 64;   // 32-wide blocks of a wave: channels, tokens
    constexpr int C16 = BK / 16, RPL = 64 / C16;      // 16-byte chunks of a row, rows of one LDS-direct load
    constexpr int LX = BM / RPL / NW, LW = BN / RPL / NW;   // such loads of a wave per stage
    constexpr int STAGE = (BM + BN) * BK;
    constexpr int SAME = 256 / BK;                    // rows in 256 bytes: all of LDS's banks
    static_assert(RPL * NW / SAME % C16 == 0, "every load stores its chunks in the same order");
    __shared__ __attribute__((aligned(1024))) uint8_t stages[NST * STAGE];
    constexpr int THREADS = NW * 64, NS = (BM + 2 * BN + THREADS - 1) / THREADS;
    __shared__ __attribute__((aligned(16))) float sc[NS * THREADS];   // token scales, channel scales, biases

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wt = KW ? 0 : wave & 1, wc = KW ? 0 : wave >> 1;
    W8Tile t;
    int s0 = 0, s1 = (p.K + 2 * BK - 1) / (2 * BK) * 2, split = 0;   // steps, in pairs
    if constexpr (MODE == EXPERTS) {
        if (!expert_tile<BM, BN>(p, t)) return;
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
    const int full = p.K / BK;
    // the step that K ends inside, or an empty one that makes up a pair: bytes past K are zeros
    auto load_tail = [&](int s, uint8_t *buf) __attribute__((always_inline)) {
        const int k = s * BK + chunk0 * 16;
#pragma unroll
        for (int j = 0; j < LX + LW; j += 4) {
            i4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = s * BK < p.K ? row16((j + i < LX ? xb : wb) + (off[j + i] - chunk0 * 16), k, p.K)
                                        : i4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<i4 *>(place(buf, j + i) + lane * 16) = v[i];
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
    if (s0 < s1) {
        // stage s is loaded by LDS-direct loads up to `direct`, then through registers
        const int direct = min(s1, full);
#pragma unroll
        for (int i = 0; i < NST; ++i)
            if (i < 2 || s0 + i < s1) load_stage(s0 + i, stages + i * STAGE);
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
    constexpr int CW = KW ? BN : BN / 2, CHUNKS = CW / 4;   // channels of a wave, their chunks in a row
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
    const bool wide = MODE == SPLIT ? (p.N & 3) == 0
                                    : (p.N & 7) == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
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
                if (n + 4 * h < n_valid) *reinterpret_cast<i4 *>(to + 4 * h) = v[h];
        } else {
            const float xs = sc[tok];
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (float)v[i / 4][i % 4] * xs * ws[i / 4][i % 4] + bs[i / 4][i % 4];
            if (n < n_valid) put8(p.y, o, f, p.y_bf16);
        }
    };
    // rows that start anywhere: value by value, neighbouring lanes neighbouring channels (623 x 23755 of K = 280
    // in 30 us; 38 with a lane's eight in turn)
    auto fetch1 = [&](const uint8_t *region, int r, int c) __attribute__((always_inline)) {
        return *reinterpret_cast<const int *>(region + r * (CW * 4) + ((c / 4 ^ (r & (CHUNKS - 1))) * 16) + c % 4 * 4);
    };
    auto emit1 = [&](int tok, int c, int v) __attribute__((always_inline)) {
        if (tok >= m_valid || c >= n_valid) return;
        const int64_t o = (int64_t)(t.first + tok) * p.N + t.n0 + c;
        if constexpr (MODE == SPLIT)
            p.part[(int64_t)split * p.rows * p.N + o] = v;
        else
            put(p.y, o, (float)v * sc[tok] * sc[BM + c] + sc[BM + BN + c], p.y_bf16);
    };
    if constexpr (KW) {
        // every wave's sums of the tile; then eight lanes add up and finish a row
#pragma unroll
        for (int b = 0; b < TT; ++b) stash(b, stages + (wave * TT + b) * REGION);
        sync(std::integral_constant<int, 0>{});
        if (wide) {
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
#pragma unroll 2
            for (int row = wave; row < BM; row += NW) {
                int v = 0;
#pragma unroll
                for (int q = 0; q < NW; ++q) v += fetch1(stages + (q * TT + row / 32) * REGION, row % 32, lane);
                emit1(row, lane, v);
            }
        }
    } else {
        uint8_t *mine = stages + wave * REGION;
        constexpr int RSTEP = 64 / (CW / 8);
#pragma unroll
        for (int b = 0; b < TT; ++b) {
            const int tok0 = (wt * TT + b) * 32;
            stash(b, mine);
            if (wide) {
#pragma unroll 4
                for (int r = lane / (CW / 8); r < 32; r += RSTEP) {
                    const i4 v[2] = {fetch(mine, r, 0), fetch(mine, r, 1)};
                    emit(tok0 + r, v);
                }
            } else {
#pragma unroll 4
                for (int i = 0; i < 32 * CW / 64; ++i) {
                    const int r = i / (CW / 64), c = i % (CW / 64) * 64 + lane;
                    emit1(tok0 + r, wc * CW + c, fetch1(mine, r, c));
                }
            }
        }
    }
}

// Sums of the splits' planes, in their order, scaled and rounded: V values of a row a thread
template <int V>
__global__ __launch_bounds__(256) void w8a8_reduce_kernel(W8Args p)
{
    const int64_t MN = (int64_t)p.rows * p.N, o = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (o >= MN) return;
    typedef int iv __attribute__((ext_vector_type(V)));
    typedef float fv __attribute__((ext_vector_type(V)));
    iv s = *reinterpret_cast<const iv *>(p.part + o);
    for (int q = 1; q < p.splits; ++q) s += *reinterpret_cast<const iv *>(p.part + q * MN + o);
    const int m = (int)(o / p.N), n = (int)(o - (int64_t)m * p.N);
    const float xs = p.xs[m];
    fv v;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = (float)s[i] * xs * p.ws[n + i];
        if (p.bias) v[i] += p.bias[n + i];
    }
    if (p.y_bf16) {
        typedef __bf16 bv __attribute__((ext_vector_type(V)));
        *reinterpret_cast<bv *>(static_cast<__bf16 *>(p.y) + o) = __builtin_convertvector(v, bv);
    } else {
        typedef _Float16 hv __attribute__((ext_vector_type(V)));
        *reinterpret_cast<hv *>(static_cast<_Float16 *>(p.y) + o) = __builtin_convertvector(v, hv);
    }
}

void reduce_launch(const W8Args &a, hipStream_t s)
{
    const int64_t MN = (int64_t)a.rows * a.N;
    if (a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 8 == 0)
        w8a8_reduce_kernel<4><<<(unsigned)((MN / 4 + 255) / 256), 256, 0, s>>>(a);
    else
        w8a8_reduce_kernel<1><<<(unsigned)((MN + 255) / 256), 256, 0, s>>>(a);
}

}  // namespace

namespace {

template <int U, bool LOOP, bool GROUPED>
void stream_launch(const W8Args &a, hipStream_t s)
{
    w8a8_stream_kernel<U, LOOP, GROUPED><<<dim3((a.N + 15) / 16, GROUPED ? a.E : 1), W * 64, 0, s>>>(a);
}

template <bool GROUPED>
void stream(const W8Args &a, hipStream_t s)
{
    const int units = a.K / 128;
    if (units <= W)
        stream_launch<1, false, GROUPED>(a, s);
    else if (units <= 2 * W)
        stream_launch<2, false, GROUPED>(a, s);
    else if (units <= 4 * W)
        stream_launch<4, false, GROUPED>(a, s);
    else
        stream_launch<2, true, GROUPED>(a, s);
}

constexpr int kCUs = 256;

template <int B, int NW, W8Mode MODE>
void tile_launch(const W8Args &a, int64_t tiles, hipStream_t s)
{
    w8a8_tile_kernel<B, B, NW, MODE><<<(unsigned)round_up(tiles, 8), NW * 64, 0, s>>>(a);
}

template <W8Mode MODE>
void tile_launch(const W8Args &a, int size, int64_t tiles, hipStream_t s)
{
    if (size == 64 && tiles <= kCUs)
        tile_launch<64, 8, MODE>(a, tiles, s);
    else if (size == 64)
        tile_launch<64, 4, MODE>(a, tiles, s);
    else if (size == 128)
        tile_launch<128, 4, MODE>(a, tiles, s);
    else
        tile_launch<256, 4, MODE>(a, tiles, s);
}

// Rows up to which a dense product streams the weights: one pass serves 16.
constexpr int kStreamRows = 16;

struct W8Plan {
    int size, splits;                                 // tile, workgroups that share K
    int64_t tiles;
};

// workgroups of one launch: a grid holds fewer than 2^32 threads
constexpr int64_t kMaxTiles = (int64_t)1 << 23;

// The tile size and split with the least estimated time: a start and an end,
// then per 128 bytes of K a time for each tile a CU has to take (one tile of
// 64 x 64 does not fill a CU).  A split adds the pass over the partial sums.
W8Plan w8_plan(int rows, int N, int K)
{
    struct Cost {
        int size;
        double ends, step, least;                     // microseconds
    };
    constexpr Cost kCosts[] = {{64, 5.5, 0.25, 0.15}, {128, 6.0, 0.56, 0.56}, {256, 14.0, 1.6, 1.6}};
    const int pairs = (K + 255) / 256;
    W8Plan best = {64, 1, 0};
    double time = -1.0;
    for (const Cost &c : kCosts) {
        const int64_t tiles = (((int64_t)rows + c.size - 1) / c.size) * (((int64_t)N + c.size - 1) / c.size);
        if (tiles >= kMaxTiles && c.size < 256) continue;
        for (int splits = 1; splits <= 8 && (splits == 1 || splits * 2 <= pairs); splits *= 2) {
            const int64_t each = (tiles * splits + kCUs - 1) / kCUs;
            const double step = each > 1 ? each * c.step : c.least;
            const double reduce = splits > 1 ? 3.0 + (double)splits * rows * N * 8 / 4e6 : 0.0;
            const double us = c.ends + (pairs + splits - 1) / splits * 2 * step + reduce;
            if (time < 0.0 || us < time) {
                time = us;
                best = {c.size, splits, tiles * splits};
            }
        }
    }
    return best;
}

}  // namespace

size_t gemm_w8a8_workspace(int M, int N, int K)
{
    if (M <= kStreamRows) return 0;
    const W8Plan pl = w8_plan(M, N, K);
    return pl.splits > 1 ? (size_t)pl.splits * M * N * sizeof(int32_t) : 0;
}

hipError_t launch_gemm_w8a8(const W8Args &args, void *ws, hipStream_t s)
{
    W8Args a = args;
    if (a.rows <= kStreamRows) {
        const int units = a.K / 128;
        if (a.rows >= 4 && a.N >= 3 * kCUs * 16 && units > 2 * W && units <= 4 * W)
            w8a8_resident_kernel<4><<<kCUs, W * 64, 0, s>>>(a);
        else
            stream<false>(a, s);
        return hipGetLastError();
    }
    const W8Plan pl = w8_plan(a.rows, a.N, a.K);
    a.splits = pl.splits;
    a.part = static_cast<int32_t *>(ws);
    if (pl.splits > 1) {
        tile_launch<SPLIT>(a, pl.size, pl.tiles, s);
        reduce_launch(a, s);
    } else {
        tile_launch<DENSE>(a, pl.size, pl.tiles, s);
    }
    return hipGetLastError();
}

// The kernel goes by the rows that an expert has on average.  Measured (us;
// streaming / tiles of 64 / 128 / 256), 128 experts of 1536 x 2048 and 8 of
// 4096 x 4096:
//   rows an expert      4                   8                   64                 256
//   128 experts   78 / 75 / 74 / 91   90 / 80 / 78 / 95   443 / 108 / 93 / 110   - / 257 / 176 / 182
//   8 experts     28 / 32 / 41 / 57   31 / 32 / 39 / 55   152 /  39 / 40 /  55   - /  78 /  76 /  59
hipError_t launch_moe_gemm_w8a8(const W8Args &a, hipStream_t s)
{
    // the rows' offsets inside x are 32-bit in the tile kernel when they are gathered
    const bool far = a.row_slot != nullptr && (int64_t)a.x_rows * a.K >= ((int64_t)1 << 32);
    if (a.rows < 6 * a.E || far) {
        stream<true>(a, s);
        return hipGetLastError();
    }
    int size = a.rows < 64 * a.E ? 64 : a.rows < 256 * a.E || a.K < 4096 ? 128 : 256;
    // an expert's last tile is not full: at most one more for each of them
    auto tiles = [&]() { return ((int64_t)a.rows / size + a.E) * (((int64_t)a.N + size - 1) / size); };
    while (tiles() >= kMaxTiles && size < 256) size *= 2;
    tile_launch<EXPERTS>(a, size, tiles(), s);
    return hipGetLastError();
}

}  // namespace lowbit
