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
constexpr int kMinPiece = 4;             // blocks that a workgroup takes at least: one for each wave

struct AttnArgs {
    KvArgs kv;
    const uint16_t *q;
    int64_t q_stride;
    int q_heads, group, window;
    float scale2;                        // scale * log2(e)
    uint16_t *y;
    int tiles;                           // row tiles of a sequence; item = sequence * tiles + tile
    int64_t over, upto;                  // sequences of over < n * group <= upto rows are this launch's
    int share;                           // 0: a workgroup takes an item's tokens whole; else pieces that they make, items aside
    float *part_o;                       // [pieces][heads][rows][dim]
    float2 *part_ml;                     // [pieces][heads][rows]: maximum and sum of each row's softmax
    int2 *parts;                         // [items]: first piece and how many, left by the first piece's workgroup
};

// What a row tile of a sequence works on
struct Span {
    KvSeq s;
    int r0, nr;                          // first row, rows (of n * group)
    int lo, hi;                          // tokens that some row sees
    int seen_lo, seen_hi;                // tokens that every row sees
    int first, end;                      // blocks of 64 tokens that some row sees
};
// rows r0 .. r0 + nr - 1 of a sequence
__device__ __forceinline__ Span attn_rows(const AttnArgs &a, const KvSeq &s, int r0, int nr)
{
    Span t;
    t.s = s;
    t.r0 = r0;
    t.nr = nr;
    const int i0 = t.r0 / a.group, i1 = (t.r0 + max(t.nr, 1) - 1) / a.group;
    const int window = a.window > 0 ? min(a.window, max(t.s.len, 1)) : max(t.s.len, 1);
    const int64_t cap = (int64_t)a.kv.width << a.kv.page_shift;
    t.hi = (int)min((int64_t)max(t.s.pos0 + i1 + 1, 0), cap);
    t.lo = max(t.s.pos0 + i0 + 1 - window, 0);
    t.seen_hi = max(t.s.pos0 + i0 + 1, 0);
    t.seen_lo = max(t.s.pos0 + i1 + 1 - window, 0);
    t.first = t.lo / kTile;
    t.end = max((t.hi + kTile - 1) / kTile, t.first);
    return t;
}
__device__ __forceinline__ Span attn_span(const AttnArgs &a, int b, int tile, int rows)
{
    const KvSeq s = kv_sequence(a.kv, b);
    const int64_t all = (int64_t)s.n * a.group;
    const bool ours = all > a.over && all <= a.upto;
    return attn_rows(a, s, tile * rows, ours ? (int)min((int64_t)rows, all - tile * rows) : 0);
}

// The items' tokens cut into pieces of equal size, so that workgroups end
// together whatever the lengths are: with `share` pieces' worth of blocks in all,
// an item of n blocks makes ceil(n / size) pieces, at most share + items of them.
// Every wave works this out for itself from the lengths, 64 items at a time.
struct Piece {
    int item, piece, first;              // the item, which of its pieces, number of its first piece
    int count, size;                     // its pieces, blocks of a piece
};
__device__ __forceinline__ int item_blocks(const AttnArgs &a, int item, int rows, bool &any)
{
    any = false;
    if (item >= a.kv.count * a.tiles) return 0;
    const Span t = attn_span(a, item / a.tiles, item % a.tiles, rows);
    any = t.nr > 0;
    return any ? t.end - t.first : 0;
}
__device__ __forceinline__ int wave_sum(int v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
// the piece of number `want`; false: there is none
__device__ __forceinline__ bool find_piece(const AttnArgs &a, int rows, int want, Piece &o)
{
    const int lane = threadIdx.x & 63, items = a.kv.count * a.tiles;
    bool any;
    int n = item_blocks(a, lane, rows, any);
    int64_t total = wave_sum(n);
    for (int base = 64; base < items; base += 64) {
        bool more;
        total += wave_sum(item_blocks(a, base + lane, rows, more));
    }
    o.size = (int)max((total + a.share - 1) / a.share, (int64_t)kMinPiece);
    int before = 0;
    for (int base = 0; base < items; base += 64) {
        if (base > 0) n = item_blocks(a, base + lane, rows, any);
        const int mine = any ? max((n + o.size - 1) / o.size, 1) : 0;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d);
            if (lane >= d) upto += v;
        }
        const int first = before + upto - mine;
        const uint64_t hit = __ballot((first <= want) & (want < first + mine));
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            o.item = base + l;
            o.first = __builtin_amdgcn_readlane(first, l);
            o.count = __builtin_amdgcn_readlane(mine, l);
            o.piece = want - o.first;
            o.size = __builtin_amdgcn_readfirstlane(o.size);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

template <bool BF16>
__device__ __forceinline__ uint16_t round_out(float v)
{
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// 4 dims of a finished row: into y where its item is one piece, else among the pieces' results
template <int D, bool BF16>
__device__ __forceinline__ void put_result(const AttnArgs &a, const Span &t, int pieces, int number, int kvh, int rows,
                                           int rr, int d, f4 v, float top, float sum)
{
    if (pieces == 1) {
        const int r = t.r0 + rr, i = r / a.group, h = r % a.group;
        const ushort4 w = {round_out<BF16>(v[0]), round_out<BF16>(v[1]), round_out<BF16>(v[2]), round_out<BF16>(v[3])};
        *reinterpret_cast<ushort4 *>(a.y + ((int64_t)(t.s.row0 + i) * a.q_heads + kvh * a.group + h) * D + d) = w;
    } else {
        const int64_t p = ((int64_t)number * a.kv.heads + kvh) * rows + rr;
        *reinterpret_cast<f4 *>(a.part_o + p * D + d) = v;
        if (d == 0) a.part_ml[p] = float2{top, sum};
    }
}

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
// 8 codes of 4 bits, minus 8: nibbles 0 and 4 of the dword (the low halves' lowest), then 1 and 5, 2 and 6, 3 and 7.  A
// nibble under the exponent of 1024 is 1024 + code in the lowest four bits, 1024 + 16 code in the next.
// `mant` is 0x64006400 in a vector register: v_and_or_b32 takes one scalar operand.
__device__ __forceinline__ h2 nibble_low(uint32_t w, uint32_t mant)
{
    const h2 v = __builtin_bit_cast(h2, (w & 0x000F000Fu) | mant);
    return v - h2{(_Float16)1032, (_Float16)1032};
}
__device__ __forceinline__ h2 nibble_high(uint32_t w, uint32_t mant)
{
    const h2 v = __builtin_bit_cast(h2, (w & 0x00F000F0u) | mant), f = {(_Float16)0.0625, (_Float16)0.0625};
    return __builtin_elementwise_fma(v, f, h2{(_Float16)-72, (_Float16)-72});
}

// One block of 64 tokens as a lane (16 j + r) loads it.  Keys: 16 bytes hold, for 8 bits, token r's dims 64 i + 16 j ..
// + 15; for 4 bits the same of tokens r and 16 + r.  Values: dim 16 m + r (and + 16 for 4 bits) of 16 tokens.
template <int FMT, int D>
struct Codes {
    static constexpr bool I8 = FMT == LOWBIT_KV_I8;
    static constexpr int N = (I8 ? 64 : 32) * D / 1024;

    // operand v of the 2 (4 bits: 4) that a lane's 16 bytes of keys hold: step v % 2 of the 64 dims, token v / 2 of the two
    static __device__ __forceinline__ h8 key_of(u4 raw, int v, uint32_t mant)
    {
        if constexpr (I8) {
            return from_bytes(raw[v * 2], raw[v * 2 + 1], (_Float16)1152);
        } else {
            const uint32_t w = raw[v];
            return join(nibble_low(w, mant), nibble_high(w, mant), nibble_low(w >> 8, mant), nibble_high(w >> 8, mant));
        }
    }
    static __device__ __forceinline__ h8 key(const u4 *raw, int block, int step, uint32_t mant)
    {
        return I8 ? key_of(raw[block * (D / 64) + step / 2], step % 2, mant)
                  : key_of(raw[block / 2 * (D / 64) + step / 2], block % 2 * 2 + step % 2, mant);
    }
    // operand of the values for 32 tokens: `high`, the other 16 dims of 4 bits
    static __device__ __forceinline__ h8 value_of(u4 w, int high, int step, uint32_t mant)
    {
        const uint32_t w0 = w[step * 2], w1 = w[step * 2 + 1];
        if constexpr (I8) return from_bytes(w0, w1, (_Float16)1152);
        return high == 0 ? join(nibble_low(w0, mant), nibble_low(w0 >> 8, mant), nibble_low(w1, mant), nibble_low(w1 >> 8, mant))
                         : join(nibble_high(w0, mant), nibble_high(w0 >> 8, mant), nibble_high(w1, mant), nibble_high(w1 >> 8, mant));
    }
    static __device__ __forceinline__ h8 value(const u4 *raw, int m, int step, uint32_t mant)
    {
        return I8 ? value_of(raw[m], 0, step, mant) : value_of(raw[m / 2], m % 2, step, mant);
    }
    // which of 4 tokens the operand has in place e
    static constexpr __device__ int order(int e) { return I8 || e % 3 == 0 ? e : 3 - e; }
};

__device__ __forceinline__ bool inside(int at, int lo, int hi) { return (at >= lo) & (at < hi); }

// largest over the four lanes of a column (l, l ^ 16, l ^ 32, l ^ 48): swaps of lane rows, no LDS
__device__ __forceinline__ float column_max(float v)
{
    auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float column_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// One block of 64 tokens in registers, as loaded
template <int FMT, int D>
struct BlockRegs {
    static constexpr bool I8 = FMT == LOWBIT_KV_I8;
    static constexpr int N = Codes<FMT, D>::N, L = I8 ? 1 : 4;
    u4 kr[N], vr[N];
    f4 ks[4], vs[4], kl[L], vl[L];

    // `part`: the head's part of the page; `at`: first token of the block in the page
    static __device__ __forceinline__ u4 get(__amdgpu_buffer_rsrc_t part, int lane_at, int at)
    {
        return __builtin_amdgcn_raw_buffer_load_b128(part, lane_at, at, 0);
    }
    __device__ __forceinline__ void load_keys(__amdgpu_buffer_rsrc_t part, int at, int lane)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) kr[i] = get(part, lane * 16, kv_code_bytes(FMT, at, D) + i * 1024);
    }
    __device__ __forceinline__ void load_values(__amdgpu_buffer_rsrc_t part, int at, int lane, int page_size)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) vr[i] = get(part, lane * 16, kv_code_bytes(FMT, page_size + at, D) + i * 1024);
    }
    __device__ __forceinline__ void load_arrays(__amdgpu_buffer_rsrc_t part, int at, int j, int page_size)
    {
        const int p = 2 * kv_code_bytes(FMT, page_size, D) + at * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            ks[q] = __builtin_bit_cast(f4, get(part, 16 * j + 64 * q, p));
            vs[q] = __builtin_bit_cast(f4, get(part, 16 * j + 64 * q, p + (I8 ? 4 : 8) * page_size));
            if constexpr (!I8) {
                kl[q] = __builtin_bit_cast(f4, get(part, 16 * j + 64 * q, p + 4 * page_size));
                vl[q] = __builtin_bit_cast(f4, get(part, 16 * j + 64 * q, p + 12 * page_size));
            }
        }
    }
};

// Exponents of base 2 by which a row's maximum may pass the one its terms are taken to before these are taken to it anew:
// p <= 2^kSlack, and the operand p * vscale * 2^(kTop - E) stays below 2^15.
constexpr float kSlack = 8.f;
constexpr int kTop = 6;

// 16 * NQ rows of an item as a wave holds them, and what they have summed up so far.  A lane's column is row 16 x + l % 16.
template <int FMT, int D, bool BF16, int NQ>
struct Rows {
    static constexpr bool I8 = FMT == LOWBIT_KV_I8;
    static constexpr int KS = D / 32, M = D / 16;
    typedef Codes<FMT, D> C;
    h8 qf[NQ][KS];
    float c[NQ], qsum[NQ];               // scale * log2(e) / (what the row's queries were multiplied by); their sum
    int see_lo[NQ], see_hi[NQ];          // tokens that the row sees
    f4 o[NQ][M];                         // sum p * vscale * 2^(kTop - E) * code, 4 dims of the lane's column
    float m[NQ], mc[NQ], l[NQ], bias[NQ];// maximum of s, that times c, sums of the lane's p and p * vmin
    int E;

    // rows r0 .. of the item, nr of them there
    __device__ __forceinline__ void load(const AttnArgs &a, const KvSeq &seq, int kvh, int r0, int nr, int lane)
    {
        const int j = lane >> 4, n = lane & 15;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int r = r0 + (x * 16 + n < nr ? x * 16 + n : 0), i = r / a.group, h = r % a.group;
            const uint16_t *src = a.q + (int64_t)(seq.row0 + i) * a.q_stride + (kvh * a.group + h) * D + 16 * j;
            see_hi[x] = seq.pos0 + i + 1;
            see_lo[x] = a.window > 0 ? see_hi[x] - min(a.window, max(seq.len, 1)) : 0;
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
                qsum[x] = column_sum(qsum[x]);
            }
#pragma unroll
            for (int i = 0; i < M; ++i) o[x][i] = f4{0.f, 0.f, 0.f, 0.f};
            m[x] = -INFINITY;
            mc[x] = l[x] = bias[x] = 0.f;
        }
        E = -100;
    }

    // s: products of the queries with a block's codes (tokens 16 q + 4 j + e); leaves the operand of the product with its
    // values.  kl, vl (4 bits): minima + 8 scales.  masked: some row does not see all of the block, whose first token is
    // t0; it has tokens that some row sees in [some_lo, some_hi).
    __device__ __forceinline__ void weigh(f4 (&s)[NQ][4], const f4 (&ks)[4], const f4 *kl, f4 (&vs)[4], f4 *vl,
                                          bool masked, bool paged, int64_t t0, int some_lo, int some_hi, int j,
                                          h8 (&pf)[NQ][2])
    {
        if (masked) {
            // tokens that no row sees: their scales do not count
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 16 * q + 4 * j + e;
                    vs[q][e] = inside(at, some_lo, some_hi) ? vs[q][e] : 0.f;
                }
        }
        // value scales: the largest exponent so far, infinities and NaN aside
        float v_top = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; e += 2)       // as fmaxf would, without quieting what was loaded first
                asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(v_top) : "v"(vs[q][e]), "v"(vs[q][e + 1]));
        v_top = column_max(v_top);
        if ((uint32_t)__builtin_amdgcn_readfirstlane(__float_as_uint(v_top)) >= 0x7f800000u) {
            v_top = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w = fabsf(vs[q][e]);
                    v_top = w <= FLT_MAX ? fmaxf(v_top, w) : v_top;
                }
            v_top = column_max(v_top);
        }
        const int e_new = max((int)((uint32_t)__builtin_amdgcn_readfirstlane(__float_as_uint(v_top)) >> 23) - 127, E);
        const float v_norm = ldexpf(1.f, kTop - e_new);
        if (e_new != E) {
            const float f = ldexpf(1.f, E - e_new);
#pragma unroll
            for (int x = 0; x < NQ; ++x)
#pragma unroll
                for (int i = 0; i < M; ++i) o[x][i] *= f;
            E = e_new;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) vs[q] *= v_norm;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[x][q][e] *= ks[q][e];
                    if constexpr (!I8) s[x][q][e] = __builtin_fmaf(kl[q][e], qsum[x], s[x][q][e]);
                }
            // tokens of the block that the lane's row sees, from its own first
            int lo = 0, hi = kTile;
            if (masked) {
                lo = (int)min(max((int64_t)see_lo[x] - t0, (int64_t)0), (int64_t)kTile) - 4 * j;
                hi = (paged ? (int)min(max((int64_t)see_hi[x] - t0, (int64_t)0), (int64_t)kTile) : 0) - 4 * j;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[x][q][e] = inside(16 * q + e, lo, hi) ? s[x][q][e] : -INFINITY;
            }
            float top = m[x];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, s[x][q][e]);
            // the maximum moves where a row's first token is seen, and where it has grown by more than the slack
            const bool far = m[x] == -INFINITY ? top != -INFINITY : __builtin_fmaf(top, c[x], -mc[x]) > kSlack;
            if (__any(far)) {
                top = column_max(top);
                const float ref = top == -INFINITY ? 0.f : top * c[x];
                const float alpha = m[x] == -INFINITY ? 0.f : exp2_fast(mc[x] - ref);
                l[x] *= alpha;
                bias[x] *= alpha;
#pragma unroll
                for (int i = 0; i < M; ++i) o[x][i] *= alpha;
                m[x] = top;
                mc[x] = ref;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = exp2_fast(__builtin_fmaf(s[x][q][e], c[x], -mc[x]));
                    l[x] += p;
                    s[x][q][e] = p;
                }
            // a token that is not seen has p = 0, and counts for nothing even where its scale is no number
            if constexpr (!I8) {
                if (masked) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bias[x] += inside(16 * q + e, lo, hi) ? s[x][q][e] * vl[q][e] : 0.f;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) bias[x] = __builtin_fmaf(s[x][q][e], vl[q][e], bias[x]);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[x][q][e] *= vs[q][e];
            if (masked)
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[x][q][e] = inside(16 * q + e, lo, hi) ? s[x][q][e] : 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) pf[x][e / 8][e % 8] = (_Float16)s[x][e / 4][C::order(e % 4)];
        }
    }
};

// Few rows: a workgroup of W waves has the 16 * NQ rows of an item, and each wave every W-th block of tokens of its
// piece.  A block's loads are under way while the one before is worked on: its keys are asked for as soon as the last
// product with the keys before them has begun, scales and values likewise, so that they need no registers of their own.
template <int FMT, int D, bool BF16, int NQ, int W>
__global__ __launch_bounds__(W * 64, D * NQ > 128 ? 1 : 2) void kv_attention_kernel(AttnArgs a)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    constexpr int ROWS = 16 * NQ, KS = D / 32, M = D / 16, DH = D < 128 ? D : 128, LD = DH + 4;
    typedef Codes<FMT, D> C;
    __shared__ __attribute__((aligned(16))) float o_s[W * 16 * LD];
    __shared__ float m_s[W][16], l_s[W][16], b_s[W][16];
    __shared__ int e_s[W];

    const int kvh = blockIdx.x % a.kv.heads, number = blockIdx.x / a.kv.heads;
    Piece pc = {number, 0, 0, 1, 0};
    if (a.share > 0 && !find_piece(a, ROWS, number, pc)) return;
    const int item = __builtin_amdgcn_readfirstlane(pc.item), b = item / a.tiles;
    const Span t = attn_span(a, b, item % a.tiles, ROWS);
    if (t.nr <= 0) return;
    if (a.share > 0 && pc.piece == 0 && kvh == 0 && threadIdx.x == 0) a.parts[item] = int2{pc.first, pc.count};
    const int begin = __builtin_amdgcn_readfirstlane(t.first + pc.piece * pc.size);
    const int end = __builtin_amdgcn_readfirstlane(pc.count > 1 ? min(begin + pc.size, t.end) : t.end);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane >> 4, n = lane & 15;

    // the wave's blocks: begin + wave + W * i, i < turns; the pages of 64 of them at a time, one a lane
    const int turns = (max(end - begin - wave, 0) + W - 1) / W;
    auto pages_of = [&](int i) {
        const int blk = begin + wave + W * (i + lane);
        return blk < end ? kv_page(a.kv, b, blk) : -1;
    };
    int pages = pages_of(0);
    Rows<FMT, D, BF16, NQ> w;
    w.load(a, t.s, kvh, t.r0, t.nr, lane);

    const int page_size = 1 << a.kv.page_shift;
    BlockRegs<FMT, D> r;
    int blk = begin + wave, page = __builtin_amdgcn_readlane(pages, 0);
    // a block without a page is read from page 0 and not seen
    auto part_of = [&](int p) { return buffer_rsrc(kv_part(a.kv, max(p, 0), kvh), a.kv.part); };
    uint32_t mant = 0x64006400u;
    asm("" : "+v"(mant));

    // `more`: another block follows
    auto step = [&](auto more, __amdgpu_buffer_rsrc_t part, int next_at) {
        constexpr bool MORE = decltype(more)::value;
        f4 s[NQ][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x][q] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const h8 kf = C::key(r.kr, q, k, mant);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
                    s[x][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, w.qf[x][k], s[x][q], 0, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MORE) r.load_keys(part, next_at, lane);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!I8) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r.kl[q][e] = __builtin_fmaf(8.f, r.ks[q][e], r.kl[q][e]);
                    r.vl[q][e] = __builtin_fmaf(8.f, r.vs[q][e], r.vl[q][e]);
                }
        }
        const int64_t t0 = (int64_t)blk * kTile;
        const bool masked = page < 0 || blk < (t.seen_lo + kTile - 1) / kTile || blk >= t.seen_hi / kTile;
        h8 pf[NQ][2];
        w.weigh(s, r.ks, r.kl, r.vs, r.vl, masked, page >= 0, t0, (int)max((int64_t)0, t.lo - t0),
                page < 0 ? 0 : (int)min((int64_t)kTile, t.hi - t0), j, pf);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MORE) r.load_arrays(part, next_at, j, page_size);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const h8 vf = C::value(r.vr, i, u, mant);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
                    w.o[x][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[x][u], w.o[x][i], 0, 0, 0);
            }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MORE) r.load_values(part, next_at, lane, page_size);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (turns > 0) {
        {
            const auto part = part_of(page);
            const int at = (blk * kTile) & (page_size - 1);
            r.load_keys(part, at, lane);
            r.load_arrays(part, at, j, page_size);
            r.load_values(part, at, lane, page_size);
        }
        for (int i = 0; i + 1 < turns; ++i) {
            if ((i & 63) == 63) pages = pages_of(i + 1);
            const int next_page = __builtin_amdgcn_readlane(pages, (i + 1) & 63);
            step(std::true_type{}, part_of(next_page), ((blk + W) * kTile) & (page_size - 1));
            page = next_page;
            blk += W;
        }
        step(std::false_type{}, part_of(page), 0);
    }

    // the waves' results joined, 16 rows and up to 128 dims at a time
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        w.l[x] = column_sum(w.l[x]);
        w.bias[x] = column_sum(w.bias[x]);
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += DH) {
            if (x > 0 || d0 > 0) __syncthreads();
            if (j == 0) {
                m_s[wave][n] = w.mc[x];
                l_s[wave][n] = w.l[x];
                b_s[wave][n] = w.bias[x];
                if (n == 0) e_s[wave] = w.E - kTop;
            }
#pragma unroll
            for (int i = 0; i < DH / 16; ++i)
                *reinterpret_cast<f4 *>(o_s + (wave * 16 + n) * LD + 16 * i + 4 * j) = w.o[x][d0 / 16 + i];
            __syncthreads();
            for (int at = threadIdx.x; at < 16 * DH / 4; at += W * 64) {
                const int row = at / (DH / 4), d = at % (DH / 4) * 4, rr = x * 16 + row;
                if (rr >= t.nr) continue;
                float top = -INFINITY, sum = 0.f, f[W];
#pragma unroll
                for (int q = 0; q < W; ++q) top = l_s[q][row] == 0.f ? top : fmaxf(top, m_s[q][row]);
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    f[q] = l_s[q][row] == 0.f ? 0.f : exp2_fast(m_s[q][row] - top);
                    sum += f[q] * l_s[q][row];
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    if (l_s[q][row] == 0.f) continue;
                    const f4 ow = *reinterpret_cast<const f4 *>(o_s + (q * 16 + row) * LD + d);
                    const float g = f[q] * inv;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += ldexpf(ow[e] * g, e_s[q]) + b_s[q][row] * g;
                }
                put_result<D, BF16>(a, t, pc.count, number, kvh, ROWS, rr, d0 + d, v, top, sum);
            }
        }
    }
}

// Many rows: a workgroup of W waves has 16 * NQ rows of an item in each, and takes the blocks of its piece one by one.
// Codes become fp16 operands once for all waves and lie in LDS in the order in which a wave reads them, 16 bytes a lane:
// no bank conflicts, and no permutation.  Two buffers and one barrier a block: a block is unpacked while the one before is
// worked on, and the codes of the one after are on their way.
template <int FMT, int D, bool BF16, int NQ, int W>
__global__ __launch_bounds__(W * 64, D > 128 ? 1 : 2) void kv_attention_tile_kernel(AttnArgs a)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    constexpr int ROWS = 16 * NQ * W, KS = D / 32, M = D / 16, A = I8 ? 1 : 2;
    typedef Codes<FMT, D> C;
    constexpr int CHUNKS = 2 * C::N, MINE = (CHUNKS + W - 1) / W;
    constexpr int KFRAGS = 4 * KS, FRAGS = KFRAGS + 2 * M;        // 1 KiB each
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    h8 *frags = reinterpret_cast<h8 *>(lds);                      // [2][FRAGS][64]
    float *arrays = reinterpret_cast<float *>(lds + 2 * FRAGS * 1024);   // [2][K, V][scale, minimum][64]

    const int kvh = blockIdx.x % a.kv.heads, number = blockIdx.x / a.kv.heads;
    Piece pc = {number, 0, 0, 1, 0};
    if (a.share > 0 && !find_piece(a, ROWS, number, pc)) return;
    const int item = __builtin_amdgcn_readfirstlane(pc.item), b = item / a.tiles;
    const Span t = attn_span(a, b, item % a.tiles, ROWS);
    if (t.nr <= 0) return;
    if (a.share > 0 && pc.piece == 0 && kvh == 0 && threadIdx.x == 0) a.parts[item] = int2{pc.first, pc.count};
    const int begin = __builtin_amdgcn_readfirstlane(t.first + pc.piece * pc.size);
    const int end = __builtin_amdgcn_readfirstlane(pc.count > 1 ? min(begin + pc.size, t.end) : t.end);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane >> 4, n = lane & 15;
    const int page_size = 1 << a.kv.page_shift;
    // the wave's own rows, and what they see
    const int w0 = wave * 16 * NQ, wn = min(t.nr - w0, 16 * NQ);
    const Span ws = attn_rows(a, t.s, t.r0 + w0, wn);

    auto pages_of = [&](int blk) { return blk + lane < end ? kv_page(a.kv, b, blk + lane) : -1; };
    int pages = pages_of(begin);
    Rows<FMT, D, BF16, NQ> w;
    w.load(a, t.s, kvh, wn > 0 ? t.r0 + w0 : t.r0, wn, lane);
    uint32_t mant = 0x64006400u;
    asm("" : "+v"(mant));

    // codes and scales of a block on their way to LDS
    u4 raw[MINE];
    float scale = 0.f, low = 0.f;
    int page_in = -1;                    // page of the block in raw
    auto fetch = [&](int blk) {
        const int i = blk - begin;
        if ((i & 63) == 0 && i > 0) pages = pages_of(blk);
        page_in = __builtin_amdgcn_readlane(pages, i & 63);
        const auto part = buffer_rsrc(kv_part(a.kv, max(page_in, 0), kvh), a.kv.part);
        const int at = (blk * kTile) & (page_size - 1);
#pragma unroll
        for (int q = 0; q < MINE; ++q) {
            const int chunk = wave + q * W;
            const int from = chunk < C::N ? kv_code_bytes(FMT, at, D) + chunk * 1024
                                          : kv_code_bytes(FMT, page_size + at, D) + (chunk - C::N) * 1024;
            if (chunk < CHUNKS) raw[q] = BlockRegs<FMT, D>::get(part, lane * 16, from);
        }
        if (wave < 2) {
            const int from = 2 * kv_code_bytes(FMT, page_size, D) + at * 4 + wave * A * page_size * 4;
            scale = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part, lane * 4, from, 0));
            if constexpr (!I8)
                low = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part, lane * 4, from + page_size * 4, 0));
        }
    };
    auto unpack = [&](int buf) {
        h8 *to = frags + buf * FRAGS * 64 + lane;
#pragma unroll
        for (int q = 0; q < MINE; ++q) {
            const int chunk = wave + q * W;
            if (chunk >= CHUNKS) break;
            if (chunk < C::N) {
                // keys: for 8 bits 16 tokens' 64 dims, two steps; for 4 bits those of 32 tokens
                const int i = chunk % (D / 64), q0 = chunk / (D / 64) * (I8 ? 1 : 2);
#pragma unroll
                for (int v = 0; v < (I8 ? 2 : 4); ++v)
                    to[((q0 + v / 2) * KS + 2 * i + v % 2) * 64] = C::key_of(raw[q], v, mant);
            } else {
                // values: 16 (32) dims, two steps of 32 tokens
                const int i = (chunk - C::N) * (I8 ? 1 : 2);
#pragma unroll
                for (int v = 0; v < (I8 ? 2 : 4); ++v)
                    to[(KFRAGS + (i + v / 2) * 2 + v % 2) * 64] = C::value_of(raw[q], v / 2, v % 2, mant);
            }
        }
        if (wave < 2) {
            float *at = arrays + ((buf * 2 + wave) * A) * 64 + lane;
            at[0] = scale;
            if constexpr (!I8) at[64] = __builtin_fmaf(8.f, scale, low);
        }
    };

    int page_next = -1;
    if (begin < end) {
        fetch(begin);
        unpack(0);
        page_next = page_in;
        if (begin + 1 < end) fetch(begin + 1);
    }
    for (int blk = begin; blk < end; ++blk) {
        const int buf = (blk - begin) & 1, page = page_next;
        __syncthreads();
        if (blk + 1 < end) {
            unpack(buf ^ 1);
            page_next = page_in;
            if (blk + 2 < end) fetch(blk + 2);
        }
        if (wn <= 0 || blk < ws.first || blk >= ws.end || page < 0) continue;     // none of the wave's rows sees it
        const h8 *f = frags + buf * FRAGS * 64 + lane;
        f4 s[NQ][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x][q] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const h8 kf = f[(q * KS + k) * 64];
#pragma unroll
                for (int x = 0; x < NQ; ++x)
                    s[x][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, w.qf[x][k], s[x][q], 0, 0, 0);
            }
        }
        f4 ks[4], vs[4], kl[4], vl[4];
        const float *ar = arrays + buf * 2 * A * 64 + 4 * j;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            ks[q] = *reinterpret_cast<const f4 *>(ar + 16 * q);
            vs[q] = *reinterpret_cast<const f4 *>(ar + A * 64 + 16 * q);
            if constexpr (!I8) {
                kl[q] = *reinterpret_cast<const f4 *>(ar + 64 + 16 * q);
                vl[q] = *reinterpret_cast<const f4 *>(ar + 3 * 64 + 16 * q);
            }
        }
        const int64_t t0 = (int64_t)blk * kTile;
        const bool masked = blk < (ws.seen_lo + kTile - 1) / kTile || blk >= ws.seen_hi / kTile;
        h8 pf[NQ][2];
        w.weigh(s, ks, kl, vs, vl, masked, true, t0, (int)max((int64_t)0, ws.lo - t0),
                (int)min((int64_t)kTile, ws.hi - t0), j, pf);
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const h8 vf = f[(KFRAGS + i * 2 + u) * 64];
#pragma unroll
                for (int x = 0; x < NQ; ++x)
                    w.o[x][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[x][u], w.o[x][i], 0, 0, 0);
            }
    }

#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        w.l[x] = column_sum(w.l[x]);
        w.bias[x] = column_sum(w.bias[x]);
        if (x * 16 + n >= wn) continue;
        const float inv = w.l[x] == 0.f ? 0.f : 1.f / w.l[x], add = w.bias[x] * inv;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            f4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = ldexpf(w.o[x][i][e] * inv, w.E - kTop) + add;
            put_result<D, BF16>(a, t, pc.count, number, kvh, ROWS, w0 + x * 16 + n, 16 * i + 4 * j, v, w.mc[x], w.l[x]);
        }
    }
}

// The pieces of a row joined: each has its own normalised result, and weighs sum * 2^maximum.  A workgroup takes one row
// of one head, dim / 4 lanes for each of its pieces, 256 / (dim / 4) pieces at a time.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void kv_attention_join_kernel(AttnArgs a, int rows, int most)
{
    constexpr int LANES = D / 4, G = 256 / LANES;
    __shared__ f4 part[G][LANES];
    __shared__ float sums[G];
    const int rr = blockIdx.x % most, kvh = blockIdx.x / most % a.kv.heads, item = blockIdx.x / most / a.kv.heads;
    const Span t = attn_span(a, item / a.tiles, item % a.tiles, rows);
    if (rr >= t.nr) return;
    const int2 pc = a.parts[item];                    // first piece, pieces
    if (pc.y <= 1) return;
    const int64_t step = (int64_t)a.kv.heads * rows, first = ((int64_t)pc.x * a.kv.heads + kvh) * rows + rr;
    const int lane = threadIdx.x & 63, g = threadIdx.x / LANES, d = threadIdx.x % LANES * 4;
    float top = -INFINITY;
    for (int i = lane; i < pc.y; i += 64) {
        const float2 ml = a.part_ml[first + i * step];
        if (ml.y != 0.f) top = fmaxf(top, ml.x);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    f4 v = {0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
#pragma unroll 4
    for (int i = g; i < pc.y; i += G) {
        const float2 ml = a.part_ml[first + i * step];
        const f4 o = *reinterpret_cast<const f4 *>(a.part_o + (first + i * step) * D + d);
        const float f = ml.y == 0.f ? 0.f : ml.y * exp2_fast(ml.x - top);
        sum += f;
        v += o * f;
    }
    part[g][threadIdx.x % LANES] = v;
    if (d == 0) sums[g] = sum;
    __syncthreads();
    if (threadIdx.x >= LANES) return;
    v = f4{0.f, 0.f, 0.f, 0.f};
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        v += part[i][threadIdx.x];
        sum += sums[i];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int r = t.r0 + rr, i = r / a.group, h = r % a.group;
    uint16_t *to = a.y + ((int64_t)(t.s.row0 + i) * a.q_heads + kvh * a.group + h) * D + d;
    const ushort4 w4 = {round_out<BF16>(v[0] * inv), round_out<BF16>(v[1] * inv), round_out<BF16>(v[2] * inv),
                        round_out<BF16>(v[3] * inv)};
    *reinterpret_cast<ushort4 *>(to) = w4;
}

constexpr int kWaves = 4;

// A launch over the sequences of over < rows * group <= upto
struct AttnPlan {
    bool tile;
    int nq, waves, rows;                 // 16 * nq rows for all waves (few) or for each (tile)
    int64_t over, upto, pieces;          // workgroups for each head
    int tiles, share;
};
int64_t plan_bytes(const AttnPlan &p, const KvArgs &a)
{
    if (p.share == 0) return 0;
    return p.pieces * a.heads * p.rows * (a.dim * 4 + 8) + round_up((int64_t)p.tiles * a.count * 8, 256);
}
void cut_plan(AttnPlan &p, const KvArgs &a, int64_t most_rows, int slots, int min_piece)
{
    p.tiles = (int)((most_rows + p.rows - 1) / p.rows);
    const int64_t items = (int64_t)p.tiles * a.count, blocks = ((int64_t)a.width << a.page_shift) / kTile;
    const bool cut = items * a.heads < slots * (p.tile ? 1 : 4) && items <= 1024 && blocks > min_piece;
    p.share = cut ? std::max(slots / a.heads, 1) : 0;
    p.pieces = cut ? std::min(items + p.share, items * ((blocks + min_piece - 1) / min_piece)) : items;
}
constexpr int64_t kFewRows = 32, kFewBeside = 16;
// one launch or two: sequences of many rows first
int attn_plan(const KvArgs &a, int q_heads, AttnPlan *p)
{
    const int64_t rows = (int64_t)a.max_rows * (q_heads / a.heads);
    int n = 0;
    const int64_t few = kFewRows;
    if (rows > few) {
        AttnPlan &t = p[n++];
        t.tile = true;
        t.nq = a.dim == 256 ? 1 : 2;
        t.waves = 8;
        t.rows = 16 * t.nq * t.waves;
        t.over = a.count > 1 ? kFewBeside : 0;
        t.upto = INT64_MAX;
        cut_plan(t, a, rows, 256, kMinPiece);
        if (a.count == 1) return n;
    }
    AttnPlan &f = p[n++];
    f.tile = false;
    const int64_t most = rows > few ? kFewBeside : rows;
    f.nq = most <= 16 ? 1 : 2;
    f.waves = kWaves;
    f.rows = 16 * f.nq;
    f.over = 0;
    f.upto = rows > few ? kFewBeside : INT64_MAX;
    cut_plan(f, a, most, a.dim * f.nq > 128 ? 256 : 512, kMinPiece);
    return n;
}

}  // namespace

bool kv_attention_fits(const KvArgs &a, int q_heads)
{
    const int64_t rows = (int64_t)a.max_rows * (q_heads / a.heads);
    if (rows >= ((int64_t)1 << 31) - 4096) return false;
    AttnPlan p[2];
    const int n = attn_plan(a, q_heads, p);
    for (int i = 0; i < n; ++i)
        if ((int64_t)p[i].tiles * a.count >= ((int64_t)1 << 22) || p[i].pieces * a.heads >= ((int64_t)1 << 22) ||
            (int64_t)p[i].tiles * a.count * a.heads * p[i].rows >= ((int64_t)1 << 31))
            return false;
    return true;
}

size_t kv_attention_workspace(const KvArgs &a, int q_heads)
{
    AttnPlan p[2];
    const int n = attn_plan(a, q_heads, p);
    int64_t most = 0;
    for (int i = 0; i < n; ++i) most = std::max(most, plan_bytes(p[i], a));
    return (size_t)most;
}

hipError_t launch_kv_attention(const KvArgs &kv, const void *q, int64_t q_stride, int q_heads, int bf16, float scale,
                               int window, void *y, void *ws, hipStream_t s)
{
    AttnPlan plans[2];
    const int n = attn_plan(kv, q_heads, plans);
    auto launch = [&](const AttnPlan &p, auto fmt, auto dim, auto bf) {
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value;
        constexpr bool B = decltype(bf)::value;
        AttnArgs a{kv, static_cast<const uint16_t *>(q), q_stride, q_heads, q_heads / kv.heads, window, scale * kLog2e,
                   static_cast<uint16_t *>(y), p.tiles, p.over, p.upto, p.share, nullptr, nullptr, nullptr};
        if (p.share > 0) {
            a.part_o = static_cast<float *>(ws);
            a.part_ml = reinterpret_cast<float2 *>(a.part_o + p.pieces * kv.heads * p.rows * kv.dim);
            a.parts = reinterpret_cast<int2 *>(a.part_ml + p.pieces * kv.heads * p.rows);
        }
        const unsigned grid = (unsigned)(p.pieces * kv.heads);
        auto tile = [&](auto nq, auto waves) {
            constexpr int NQ = decltype(nq)::value, W = decltype(waves)::value;
            constexpr size_t lds = 512 * D + (F == LOWBIT_KV_I8 ? 1024 : 2048);
            auto kernel = kv_attention_tile_kernel<F, D, B, NQ, W>;
            if (lds > 65536) {
                const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                         (int)lds);
                if (e != hipSuccess) return e;
            }
            kernel<<<grid, W * 64, lds, s>>>(a);
            return hipGetLastError();
        };
        typedef std::integral_constant<int, 1> one;
        typedef std::integral_constant<int, 2> two;
        hipError_t e;
        if (p.tile) {
            typedef std::integral_constant<int, D == 256 ? 1 : 2> nq;
            e = p.waves == 8 ? tile(nq{}, std::integral_constant<int, 8>{}) : tile(nq{}, std::integral_constant<int, 4>{});
        } else {
            if (p.nq == 1) kv_attention_kernel<F, D, B, one::value, kWaves><<<grid, kWaves * 64, 0, s>>>(a);
            else kv_attention_kernel<F, D, B, two::value, kWaves><<<grid, kWaves * 64, 0, s>>>(a);
            e = hipGetLastError();
        }
        if (e != hipSuccess || p.share == 0) return e;
        const int most = (int)std::min<int64_t>(p.rows, (int64_t)kv.max_rows * a.group);
        kv_attention_join_kernel<D, B><<<(unsigned)((int64_t)kv.count * p.tiles * kv.heads * most), 256, 0, s>>>(
            a, p.rows, most);
        return hipGetLastError();
    };
    auto with_bf = [&](const AttnPlan &p, auto fmt, auto dim) {
        return bf16 ? launch(p, fmt, dim, std::true_type{}) : launch(p, fmt, dim, std::false_type{});
    };
    auto with_dim = [&](const AttnPlan &p, auto fmt) {
        return kv.dim == 64 ? with_bf(p, fmt, std::integral_constant<int, 64>{})
               : kv.dim == 128 ? with_bf(p, fmt, std::integral_constant<int, 128>{})
                               : with_bf(p, fmt, std::integral_constant<int, 256>{});
    };
    for (int i = 0; i < n; ++i) {
        const hipError_t e = kv.fmt == LOWBIT_KV_I8 ? with_dim(plans[i], std::integral_constant<int, LOWBIT_KV_I8>{})
                                                    : with_dim(plans[i], std::integral_constant<int, LOWBIT_KV_U4>{});
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lowbit
