// kv_attention.hip -- attention of new tokens over a quantised cache in pages.
//
//   y[r][h] = sum_j p_j v_j,  p = softmax_j(scale * q[r][h] . k_j)  over the tokens j that row r sees
//
// The query heads that share a key/value head and the tokens of a sequence are
// the rows of one matrix product (row = token * group + head of the group), 16
// at a time.  Both products run on v_mfma_f32_16x16x32_f16 with the cache as the
// A operand, straight from memory: the pages hold keys and values in the order of
// that operand, codes become fp16 exactly in registers (1024 + code is an fp16
// bit pattern; the bias is then subtracted).  S^T = K Q^T leaves a lane with 4
// tokens of each 16 for one query, which is the B operand of O^T = V^T P^T with
// the tokens of a 32 in the order 4j..4j+3, 16+4j..16+4j+3: the probabilities
// never leave their registers.
//
// Scales stand outside of the sums over dims (keys) and inside of those over
// tokens (values): s = kscale * acc (+ kmin * sum of q, 4 bits), and the fp16
// operand is p * vscale * 2^(14 - E), E the largest exponent of a value scale so
// far: p <= 1 keeps it under 2^15, and terms down to 2^-28 of the largest keep
// their 11 bits.  The minima of values enter as sum p * vmin, one number per row.
// The softmax runs in one pass with a running maximum.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "kv_cache.hpp"

namespace lowbit {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTile = 64;                // tokens of a step: one block of a page

struct AttnArgs {
    KvArgs kv;
    const uint16_t *q;
    int64_t q_stride;
    int q_heads, group, window;
    float scale2;                        // scale * log2(e)
    uint16_t *y;
    int tiles, splits;                   // row tiles of a sequence, workgroups that share its tokens
    float *part_o;                       // [count][tiles][heads][splits][rows][dim]
    float2 *part_ml;                     // [count][tiles][heads][splits][rows]
};

// What a row tile of a sequence works on
struct Span {
    KvSeq s;
    int r0, nr;                          // first row, rows (of n * group)
    int first, end;                      // blocks of 64 tokens that some row sees
    int lo, hi;                          // tokens that some row sees
    int seen_lo, seen_hi;                // tokens that every row sees
    int per, active;                     // blocks of a split, splits that have any
};
__device__ __forceinline__ Span attn_span(const AttnArgs &a, int b, int tile, int rows)
{
    Span t;
    t.s = kv_sequence(a.kv, b);
    t.r0 = tile * rows;
    t.nr = (int)min((int64_t)rows, (int64_t)t.s.n * a.group - t.r0);
    const int i0 = t.r0 / a.group, i1 = (t.r0 + max(t.nr, 1) - 1) / a.group;
    const int window = a.window > 0 ? min(a.window, max(t.s.len, 1)) : max(t.s.len, 1);
    const int64_t cap = (int64_t)a.kv.width << a.kv.page_shift;
    t.hi = (int)min((int64_t)max(t.s.pos0 + i1 + 1, 0), cap);
    t.lo = max(t.s.pos0 + i0 + 1 - window, 0);
    t.seen_hi = max(t.s.pos0 + i0 + 1, 0);
    t.seen_lo = max(t.s.pos0 + i1 + 1 - window, 0);
    t.first = t.lo / kTile;
    t.end = max((t.hi + kTile - 1) / kTile, t.first);
    const int n = t.end - t.first;
    t.per = max((n + a.splits - 1) / a.splits, 1);
    t.active = max((n + t.per - 1) / t.per, 1);
    return t;
}

template <bool BF16>
__device__ __forceinline__ uint16_t round_out(float v)
{
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// two codes of bytes `sel` picks, each under the fp16 exponent of 1024, minus `bias`
__device__ __forceinline__ h2 byte_pair(uint32_t w, uint32_t sel, _Float16 bias)
{
    const h2 v = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, w, sel));
    return v - h2{bias, bias};
}
__device__ __forceinline__ h8 join(h2 a, h2 b, h2 c, h2 d)
{
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ h8 from_bytes(uint32_t w0, uint32_t w1, _Float16 bias)
{
    return join(byte_pair(w0, 0x04010400u, bias), byte_pair(w0, 0x04030402u, bias),
                byte_pair(w1, 0x04010400u, bias), byte_pair(w1, 0x04030402u, bias));
}
__device__ __forceinline__ h2 nibble_pair(uint32_t w)
{
    const h2 v = __builtin_bit_cast(h2, (w & 0x000F000Fu) | 0x64006400u);
    return v - h2{(_Float16)1024, (_Float16)1024};
}

// One block of 64 tokens as a lane (16 j + r) loads it.  Keys: 16 bytes hold, for 8 bits, token r's dims 64 i + 16 j ..
// + 15; for 4 bits the same of tokens r and 16 + r.  Values: dim 16 m + r (and + 16 for 4 bits) of 16 tokens.
template <int FMT, int D>
struct Codes {
    static constexpr bool I8 = FMT == LOWBIT_KV_I8;
    static constexpr int N = (I8 ? 64 : 32) * D / 1024;

    static __device__ __forceinline__ h8 key(const u4 *raw, int block, int step)
    {
        if constexpr (I8) {
            const u4 w = raw[block * (D / 64) + step / 2];
            return from_bytes(w[step % 2 * 2], w[step % 2 * 2 + 1], (_Float16)1152);
        } else {
            const uint32_t w = raw[block / 2 * (D / 64) + step / 2][block % 2 * 2 + step % 2];
            return join(nibble_pair(w), nibble_pair(w >> 4), nibble_pair(w >> 8), nibble_pair(w >> 12));
        }
    }
    static __device__ __forceinline__ h8 value(const u4 *raw, int m, int step)
    {
        if constexpr (I8) return from_bytes(raw[m][step * 2], raw[m][step * 2 + 1], (_Float16)1152);
        const u4 w = raw[m / 2];
        const uint32_t w0 = w[step * 2] >> (m % 2 * 4), w1 = w[step * 2 + 1] >> (m % 2 * 4);
        return from_bytes(w0 & 0x0F0F0F0Fu, w1 & 0x0F0F0F0Fu, (_Float16)1024);
    }
};

// Few rows: a workgroup of W waves has 16 * NQ of them, and each wave every W-th block of tokens.
template <int FMT, int D, bool BF16, int NQ, int W>
__global__ __launch_bounds__(W * 64) void kv_attention_kernel(AttnArgs a)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    constexpr int ROWS = 16 * NQ, KS = D / 32, M = D / 16, DH = D < 128 ? D : 128, LD = DH + 4;
    typedef Codes<FMT, D> C;
    __shared__ __attribute__((aligned(16))) float o_s[W * 16 * LD];
    __shared__ float m_s[W][16], l_s[W][16], b_s[W][16];
    __shared__ int e_s[W];

    int id = blockIdx.x;
    const int kvh = id % a.kv.heads;
    id /= a.kv.heads;
    const int tile = id % a.tiles;
    id /= a.tiles;
    const int split = id % a.splits, b = id / a.splits;
    const Span t = attn_span(a, b, tile, ROWS);
    if (t.nr <= 0 || split >= t.active) return;
    const int begin = t.first + split * t.per, end = min(begin + t.per, t.end);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane >> 4, n = lane & 15;

    // queries: the lane's column is row r0 + 16 x + n
    h8 qf[NQ][KS];
    float c[NQ], qsum[NQ];
    int see_lo[NQ], see_hi[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int r = t.r0 + x * 16 + n;
        const bool have = x * 16 + n < t.nr;
        const int i = (have ? r : t.r0) / a.group, h = (have ? r : t.r0) % a.group;
        const uint16_t *src = a.q + (int64_t)(t.s.row0 + i) * a.q_stride + (kvh * a.group + h) * D + 16 * j;
        see_hi[x] = t.s.pos0 + i + 1;
        see_lo[x] = a.window > 0 ? see_hi[x] - min(a.window, max(t.s.len, 1)) : 0;
        us8 raw[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) raw[k] = *reinterpret_cast<const us8 *>(src + k / 2 * 64 + k % 2 * 8);
        c[x] = a.scale2;
        if constexpr (BF16) {
            // into fp16 after a power of two that brings the row's largest value to [2^14, 2^15)
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, (uint32_t)raw[k][e] & 0x7fffu);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            const int shift = top == 0 || top >= 0x7f80u ? 0 : 141 - (int)(top >> 7);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    qf[x][k][e] = (_Float16)ldexpf(__uint_as_float((uint32_t)raw[k][e] << 16), shift);
            c[x] = ldexpf(c[x], -shift);
        } else {
#pragma unroll
            for (int k = 0; k < KS; ++k) qf[x][k] = __builtin_bit_cast(h8, raw[k]);
        }
        c[x] = fminf(fmaxf(c[x], FLT_MIN), FLT_MAX);
        qsum[x] = 0.f;
        if constexpr (!I8) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) qsum[x] += (float)qf[x][k][e];
            qsum[x] += __shfl_xor(qsum[x], 16);
            qsum[x] += __shfl_xor(qsum[x], 32);
        }
    }

    f4 o[NQ][M];
    float m[NQ], mc[NQ], l[NQ], bias[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
#pragma unroll
        for (int i = 0; i < M; ++i) o[x][i] = f4{0.f, 0.f, 0.f, 0.f};
        m[x] = -INFINITY;
        mc[x] = l[x] = bias[x] = 0.f;
    }
    int E = -100;                                     // exponent that the value scales are taken to
    const int page_size = 1 << a.kv.page_shift;
    const int codes = kv_code_bytes(FMT, page_size, D);

    for (int blk = begin + wave; blk < end; blk += W) {
        const int page = __builtin_amdgcn_readfirstlane(kv_page(a.kv, b, blk));
        if (page < 0) continue;
        const uint8_t *part = kv_part(a.kv, page, kvh);
        const int in_page = (blk * kTile) & (page_size - 1);
        const uint8_t *kp = part + kv_code_bytes(FMT, in_page, D) + lane * 16, *vp = kp + codes;
        const float *arrays = reinterpret_cast<const float *>(part + 2 * codes) + in_page + 4 * j;
        u4 kr[C::N], vr[C::N];
        f4 ks[4], vs[4], kl[4], vl[4];
#pragma unroll
        for (int i = 0; i < C::N; ++i) kr[i] = *reinterpret_cast<const u4 *>(kp + i * 1024);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            ks[q] = *reinterpret_cast<const f4 *>(arrays + 16 * q);
            if constexpr (!I8) kl[q] = *reinterpret_cast<const f4 *>(arrays + page_size + 16 * q);
            vs[q] = *reinterpret_cast<const f4 *>(arrays + (I8 ? 1 : 2) * page_size + 16 * q);
            if constexpr (!I8) vl[q] = *reinterpret_cast<const f4 *>(arrays + 3 * page_size + 16 * q);
        }
#pragma unroll
        for (int i = 0; i < C::N; ++i) vr[i] = *reinterpret_cast<const u4 *>(vp + i * 1024);

        f4 s[NQ][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x][q] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const h8 kf = C::key(kr, q, k);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
                    s[x][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[x][k], s[x][q], 0, 0, 0);
            }
        }
        const int64_t t0 = (int64_t)blk * kTile;
        const bool whole = t0 >= t.seen_lo && t0 + kTile <= t.seen_hi;
        const int some_lo = (int)max((int64_t)0, t.lo - t0), some_hi = (int)min((int64_t)kTile, t.hi - t0);

        // value scales: the largest exponent so far, tokens that no row sees and infinities aside
        uint32_t vtop = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = __float_as_uint(vs[q][e]) & 0x7fffffffu;
                vtop = max(vtop, w < 0x7f800000u && (whole || (16 * q + 4 * j + e >= some_lo && 16 * q + 4 * j + e < some_hi)) ? w : 0u);
            }
        vtop = max(vtop, (uint32_t)__shfl_xor((int)vtop, 16));
        vtop = max(vtop, (uint32_t)__shfl_xor((int)vtop, 32));
        const int e_new = __builtin_amdgcn_readfirstlane(max((int)(vtop >> 23) - 127, E));
        const float e_scale = ldexpf(1.f, E - e_new), v_norm = ldexpf(1.f, 14 - e_new);
        const bool e_moved = e_new != E;
        E = e_new;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float top = m[x];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = s[x][q][e] * ks[q][e];
                    if constexpr (!I8) v = __builtin_fmaf(kl[q][e], qsum[x], v);
                    if (!whole) {
                        const int64_t at = t0 + 16 * q + 4 * j + e;
                        v = at >= see_lo[x] && at < see_hi[x] ? v : -INFINITY;
                    }
                    s[x][q][e] = v;
                    top = fmaxf(top, v);
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float ref = top == -INFINITY ? 0.f : top * c[x];
            const float alpha = m[x] == -INFINITY ? 0.f : exp2_fast(mc[x] - ref);
            const bool moved = top != m[x];
            m[x] = top;
            mc[x] = ref;
            if (__any(moved) || e_moved) {
                l[x] *= alpha;
                bias[x] *= alpha;
                const float f = alpha * e_scale;
#pragma unroll
                for (int i = 0; i < M; ++i) o[x][i] *= f;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = exp2_fast(__builtin_fmaf(s[x][q][e], c[x], -ref));
                    float pv = p * (vs[q][e] * v_norm), pl = 0.f;
                    if constexpr (!I8) pl = p * vl[q][e];
                    if (!whole) {
                        const int64_t at = t0 + 16 * q + 4 * j + e;
                        const bool seen = at >= see_lo[x] && at < see_hi[x];
                        pv = seen ? pv : 0.f;
                        pl = seen ? pl : 0.f;
                    }
                    l[x] += p;
                    bias[x] += pl;
                    s[x][q][e] = pv;
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            h8 pf[NQ];
#pragma unroll
            for (int x = 0; x < NQ; ++x)
#pragma unroll
                for (int e = 0; e < 8; ++e) pf[x][e] = (_Float16)s[x][2 * u + e / 4][e % 4];
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const h8 vf = C::value(vr, i, u);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
                    o[x][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[x], o[x][i], 0, 0, 0);
            }
        }
    }

    // the waves' results joined, 16 rows and up to 128 dims at a time
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        l[x] += __shfl_xor(l[x], 16);
        l[x] += __shfl_xor(l[x], 32);
        bias[x] += __shfl_xor(bias[x], 16);
        bias[x] += __shfl_xor(bias[x], 32);
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += DH) {
            if (x > 0 || d0 > 0) __syncthreads();
            if (j == 0) {
                m_s[wave][n] = mc[x];
                l_s[wave][n] = l[x];
                b_s[wave][n] = bias[x];
                if (n == 0) e_s[wave] = E - 14;
            }
#pragma unroll
            for (int i = 0; i < DH / 16; ++i)
                *reinterpret_cast<f4 *>(o_s + (wave * 16 + n) * LD + 16 * i + 4 * j) = o[x][d0 / 16 + i];
            __syncthreads();
            for (int at = threadIdx.x; at < 16 * DH / 4; at += W * 64) {
                const int row = at / (DH / 4), d = at % (DH / 4) * 4, rr = x * 16 + row;
                if (rr >= t.nr) continue;
                float top = -INFINITY, sum = 0.f, f[W];
#pragma unroll
                for (int w = 0; w < W; ++w) top = l_s[w][row] == 0.f ? top : fmaxf(top, m_s[w][row]);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    f[w] = l_s[w][row] == 0.f ? 0.f : exp2_fast(m_s[w][row] - top);
                    sum += f[w] * l_s[w][row];
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (l_s[w][row] == 0.f) continue;
                    const f4 ow = *reinterpret_cast<const f4 *>(o_s + (w * 16 + row) * LD + d);
                    const float g = f[w] * inv;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += ldexpf(ow[e] * g, e_s[w]) + b_s[w][row] * g;
                }
                if (t.active == 1) {
                    const int r = t.r0 + rr, i = r / a.group, h = r % a.group;
                    uint16_t *to = a.y + ((int64_t)(t.s.row0 + i) * a.q_heads + kvh * a.group + h) * D + d0 + d;
                    const ushort4 w4 = {round_out<BF16>(v[0]), round_out<BF16>(v[1]), round_out<BF16>(v[2]),
                                        round_out<BF16>(v[3])};
                    *reinterpret_cast<ushort4 *>(to) = w4;
                } else {
                    const int64_t p =
                        ((((int64_t)b * a.tiles + tile) * a.kv.heads + kvh) * a.splits + split) * ROWS + rr;
                    *reinterpret_cast<f4 *>(a.part_o + p * D + d0 + d) = v;
                    if (d0 + d == 0) a.part_ml[p] = float2{top, sum};
                }
            }
        }
    }
}

// The splits of a row joined: each has its own normalised result, and weighs sum * 2^top.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void kv_attention_join_kernel(AttnArgs a, int rows)
{
    constexpr int LANES = D / 4;
    const int64_t at = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    const int d = threadIdx.x % LANES * 4;
    const int rr = (int)(at % rows);
    int64_t id = at / rows;
    const int kvh = (int)(id % a.kv.heads);
    id /= a.kv.heads;
    const int tile = (int)(id % a.tiles);
    const int64_t b = id / a.tiles;
    if (b >= a.kv.count) return;
    const Span t = attn_span(a, (int)b, tile, rows);
    if (rr >= t.nr || t.active == 1) return;
    const int64_t p = ((b * a.tiles + tile) * a.kv.heads + kvh) * a.splits * rows + rr;
    float top = -INFINITY, sum = 0.f;
    for (int i = 0; i < t.active; ++i) {
        const float2 ml = a.part_ml[p + (int64_t)i * rows];
        if (ml.y != 0.f) top = fmaxf(top, ml.x);
    }
    f4 v = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < t.active; ++i) {
        const float2 ml = a.part_ml[p + (int64_t)i * rows];
        if (ml.y == 0.f) continue;
        const float f = ml.y * exp2_fast(ml.x - top);
        const f4 o = *reinterpret_cast<const f4 *>(a.part_o + (p + (int64_t)i * rows) * D + d);
        sum += f;
        v += o * f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int r = t.r0 + rr, i = r / a.group, h = r % a.group;
    uint16_t *to = a.y + ((int64_t)(t.s.row0 + i) * a.q_heads + kvh * a.group + h) * D + d;
    const ushort4 w4 = {round_out<BF16>(v[0] * inv), round_out<BF16>(v[1] * inv), round_out<BF16>(v[2] * inv),
                        round_out<BF16>(v[3] * inv)};
    *reinterpret_cast<ushort4 *>(to) = w4;
}

constexpr int kWaves = 4;

struct AttnPlan {
    int nq, tiles, splits;
};
AttnPlan attn_plan(const KvArgs &a, int q_heads)
{
    AttnPlan p;
    const int64_t rows = (int64_t)a.max_rows * (q_heads / a.heads);
    p.nq = rows <= 16 ? 1 : 2;
    p.tiles = (int)((rows + 16 * p.nq - 1) / (16 * p.nq));
    const int64_t groups = (int64_t)p.tiles * a.heads * a.count;
    const int64_t blocks = (((int64_t)a.width << a.page_shift) + kTile - 1) / kTile;
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({1024 / groups, 64, blocks / kWaves}));
    return p;
}

}  // namespace

bool kv_attention_fits(const KvArgs &a, int q_heads)
{
    const int64_t rows = (int64_t)a.max_rows * (q_heads / a.heads);
    if (rows >= ((int64_t)1 << 31) - 64) return false;
    const AttnPlan p = attn_plan(a, q_heads);
    return (int64_t)p.tiles * a.count < ((int64_t)1 << 24) &&
           (int64_t)p.tiles * a.count * a.heads * p.splits < ((int64_t)1 << 24);
}

size_t kv_attention_workspace(const KvArgs &a, int q_heads)
{
    const AttnPlan p = attn_plan(a, q_heads);
    if (p.splits == 1) return 0;
    return (size_t)a.count * p.tiles * a.heads * p.splits * 16 * p.nq * (a.dim * 4 + 8);
}

hipError_t launch_kv_attention(const KvArgs &kv, const void *q, int64_t q_stride, int q_heads, int bf16, float scale,
                               int window, void *y, void *ws, hipStream_t s)
{
    const AttnPlan p = attn_plan(kv, q_heads);
    AttnArgs a{kv, static_cast<const uint16_t *>(q), q_stride, q_heads, q_heads / kv.heads, window, scale * kLog2e,
               static_cast<uint16_t *>(y), p.tiles, p.splits, nullptr, nullptr};
    const int64_t groups = (int64_t)kv.count * p.tiles * kv.heads * p.splits, rows = 16 * p.nq;
    if (p.splits > 1) {
        a.part_o = static_cast<float *>(ws);
        a.part_ml = reinterpret_cast<float2 *>(a.part_o + groups * rows * kv.dim);
    }
    auto run = [&](auto fmt, auto dim, auto bf, auto nq) {
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value, NQ = decltype(nq)::value;
        constexpr bool B = decltype(bf)::value;
        kv_attention_kernel<F, D, B, NQ, kWaves><<<(unsigned)groups, kWaves * 64, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || p.splits == 1) return e;
        constexpr int per = 256 / (D / 4);
        const int64_t all = (int64_t)kv.count * p.tiles * kv.heads * rows;
        kv_attention_join_kernel<D, B><<<(unsigned)((all + per - 1) / per), 256, 0, s>>>(a, (int)rows);
        return hipGetLastError();
    };
    auto with_nq = [&](auto fmt, auto dim, auto bf) {
        return p.nq == 1 ? run(fmt, dim, bf, std::integral_constant<int, 1>{})
                         : run(fmt, dim, bf, std::integral_constant<int, 2>{});
    };
    auto with_bf = [&](auto fmt, auto dim) {
        return bf16 ? with_nq(fmt, dim, std::true_type{}) : with_nq(fmt, dim, std::false_type{});
    };
    auto with_dim = [&](auto fmt) {
        return kv.dim == 64 ? with_bf(fmt, std::integral_constant<int, 64>{})
               : kv.dim == 128 ? with_bf(fmt, std::integral_constant<int, 128>{})
                               : with_bf(fmt, std::integral_constant<int, 256>{});
    };
    return kv.fmt == LOWBIT_KV_I8 ? with_dim(std::integral_constant<int, LOWBIT_KV_I8>{})
                                  : with_dim(std::integral_constant<int, LOWBIT_KV_U4>{});
}

}  // namespace lowbit
