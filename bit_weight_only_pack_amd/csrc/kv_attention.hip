// kv_attention.hip -- attention of new tokens over a quantised cache in pages.
//
//   y[r][h] = sum_j p_j v_j,  p = softmax_j(scale * q[r][h] . k_j)  over the tokens j that row r sees
//
// The query heads that share a key/value head and the tokens of a sequence are
// the rows of one matrix product (row = token * group + head of the group).
// Both products run on the fp16 matrix instructions with the cache as the A
// operand: the pages hold keys and values in the order of that operand, and
// codes become fp16 exactly in registers (1024 + code is an fp16 bit pattern;
// the bias, and the code's own middle, are then subtracted).  S^T = K Q^T leaves
// a lane with 4 tokens of each 16 (32x32x16: of each 8) for one query, which is
// the B operand of O^T = V^T P^T with the tokens of a 32 in the order 4j..4j+3,
// 16+4j..16+4j+3: the weights never leave their registers.
//
// Scales stand outside of the sums over dims (keys) and inside of those over
// tokens (values): s = kscale * acc (+ kmin * sum of q, 4 bits), and the fp16
// operand is p * vscale * 2^(kTop - E), E the largest exponent of a value scale
// so far; where scales differ by more than 2^8 (bf16 results: 2^14), each row
// takes its operands to the largest of its own instead (Rows::SPREAD).  The
// minima of values enter as sum p * vmin, one number per row.  The softmax runs
// in one pass; the maximum that a row's terms are taken to, a whole exponent,
// moves only where one passes it by 2^kSlack, so that most blocks rescale
// nothing.  The operand stays under 2^(kSlack + kTop + 1) = 2^15, and terms down
// to 2^-20 of one at that maximum and scale keep all their 11 bits (fp16's least
// normal number is 2^-14).
//
// Two kernels share this.  Few rows (kv_attention_kernel) read the cache once,
// and its bytes are the bound: 562 MB of 8 bit cache for one token each of 64
// sequences of up to 8192 in 108 us, 5.2 TB/s, as fast as a large copy.  Many rows
// (kv_attention_tile_kernel) are bound by the instructions of a compute unit,
// matrix and vector ones: 515 GFLOP of a causal prompt in 0.59 to 0.61 ms, 850 to
// 870 TFLOP/s, 70 % of a large library product's rate.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "kv_cache.hpp"

namespace lowbit {

namespace {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTile = 64;                // tokens of a step: one block of a page
// Items up to which they are cut, counted as sequences times the tiles of the longest, for so many fit a wave's registers (8 a
// lane).  Past it a long item is walked whole: 1024 rows of 4 heads of 256, group 2, over 4096 tokens, 112 us beside 31 single
// rows and 206 beside 32; single rows of 512 sequences, one of 65536 tokens, 171 us, of 513 438.
constexpr int kMaxItems = 512;
constexpr int kMinPiece = 4;             // blocks that a workgroup takes at least: one for each wave

// n / d and n % d for 0 <= n < 2^31 by one product: m = ceil(2^(31 + b) / d) with 2^(b - 1) < d <= 2^b
struct Divisor {
    int d, shift;
    uint32_t m;
    __host__ Divisor(int by = 1) : d(by), shift(0), m(0)
    {
        int b = 0;
        while (((int64_t)1 << b) < by) ++b;
        if (by > 1) {
            shift = b - 1;
            m = (uint32_t)((((uint64_t)1 << (31 + b)) + by - 1) / by);
        }
    }
    __device__ __forceinline__ int of(int n) const { return d == 1 ? n : (int)(__umulhi((uint32_t)n, m) >> shift); }
    __device__ __forceinline__ int rest(int n) const { return n - of(n) * d; }
};

struct AttnArgs {
    KvArgs kv;
    const uint16_t *q;
    int64_t q_stride;
    int q_heads, group, window;
    float scale2;                        // scale * log2(e)
    uint16_t *y;
    Divisor by_group, by_tiles, by_heads;
    int tiles;                           // row tiles of a sequence; item = sequence * tiles + tile
    int64_t over, upto;                  // sequences of over < n * group <= upto rows are this launch's
    int share, fill;                     // 0: a workgroup takes an item's tokens whole; else how many pieces to make of all
    float *part_o;                       // [slots][heads][rows][dim]
    float2 *part_ml;                     // [slots][heads][rows]: exponent and sum of each row's softmax
    int4 *cuts;                          // [0]: how many items are cut; then item, first slot and pieces of each
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
    const int i0 = a.by_group.of(t.r0), i1 = a.by_group.of(t.r0 + max(t.nr, 1) - 1);
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

// The items' tokens cut into pieces of equal size, so that workgroups end together whatever the lengths are.  An item of n
// blocks makes ceil(n / size) pieces, so `there` items of T blocks in all make about T / size + there / 2.  Few rows, bound
// by memory: T / size as many as are resident at once, or twice that where many items leave odd ends.  Tiles, bound by the
// compute units: pieces to fill these once, or a whole number of times, and those of an item are then made alike (a chunk of
// 1024 tokens over 4096, 4 heads of 256: 70 us for 72; few rows beside it: 44 for 36, as odd ends fill what is left), once
// more where the odd ends alone nearly do (8 heads of 64, 50 rows over 131072 tokens beside 125 times 50 over 1024: 195 us,
// 2918 with a piece of everything).  Nothing is cut where no item is much longer than a piece.  Those of items that are cut, at most 2 T / size, have slots for
// their results.  Every wave works this out for itself from the lengths, 64 items at a time, the last tiles of a sequence,
// its longest, first.
struct Piece {
    int item, piece;                     // the item, which of its pieces
    int count, size;                     // its pieces, blocks of a piece
    int slot;                            // slot of its first piece
    int cut, cuts;                       // which of the items that are cut, how many there are
};
__device__ __forceinline__ int item_blocks(const AttnArgs &a, int item, int rows)
{
    if (item < 0) return -1;
    const Span t = attn_span(a, a.by_tiles.of(item), a.by_tiles.rest(item), rows);
    return t.nr > 0 ? t.end - t.first : -1;
}
// f over the lanes below and the lane's own: within rows of 16, then row by row (0 is the identity)
template <typename F>
__device__ __forceinline__ int wave_scan(int v, F f)
{
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
    return f(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
}
__device__ __forceinline__ int plus(int p, int q) { return p + q; }
__device__ __forceinline__ int larger(int p, int q) { return max(p, q); }

// the piece of number `want`; false: there is none
__device__ __forceinline__ bool find_piece(const AttnArgs &a, int rows, int want, Piece &o)
{
    constexpr int CHUNKS = kMaxItems / 64;
    const int lane = threadIdx.x & 63, items = a.kv.count * a.tiles;
    int n[CHUNKS], most = 0, there = 0;
    uint32_t total = 0;                              // in fours: an item has up to 2^24 blocks
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        n[c] = c * 64 < items ? item_blocks(a, items - 1 - c * 64 - lane, rows) : -1;
        total += (uint32_t)(max(n[c], 0) + 3) >> 2;
        most = max(most, n[c]);
        there += __popcll(__ballot(n[c] >= 0));
    }
    total = (uint32_t)__builtin_amdgcn_readlane(wave_scan((int)total, plus), 63);
    most = __builtin_amdgcn_readlane(wave_scan(most, larger), 63);
    int wanted = there > a.share / 2 ? 2 * a.share : a.share;
    if (a.fill) {
        wanted = (there / 2 / a.share + 1) * a.share - there / 2;
        if (wanted * 2 < a.share) wanted += a.share;     // so few would make a piece of everything
    }
    const int64_t share = (((int64_t)total << 2) + wanted - 1) / wanted;
    const int even = (int)min(max(share, (int64_t)kMinPiece), (int64_t)1 << 25);     // past any item's blocks
    o.size = __builtin_amdgcn_readfirstlane(most <= even + even / 2 ? max(most, 1) : even);
    int before = 0, slots = 0;
    o.cuts = 0;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) o.cuts += __popcll(__ballot(n[c] > o.size));
    o.cut = 0;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        if (c * 64 >= items) break;
        const uint64_t cut = __ballot(n[c] > o.size);
        const int mine = n[c] < 0 ? 0 : max((n[c] + o.size - 1) / o.size, 1), kept = mine > 1 ? mine : 0;
        const int upto = wave_scan(mine, plus), kept_upto = wave_scan(kept, plus);
        const int first = before + upto - mine;
        const uint64_t hit = __ballot((first <= want) & (want < first + mine));
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            o.item = items - 1 - c * 64 - l;
            o.piece = want - __builtin_amdgcn_readlane(first, l);
            o.count = __builtin_amdgcn_readlane(mine, l);
            if (a.fill) o.size = (__builtin_amdgcn_readlane(n[c], l) + o.count - 1) / o.count;   // as many, alike
            o.slot = __builtin_amdgcn_readlane(slots + kept_upto - kept, l);
            o.cut += __popcll(cut & (((uint64_t)1 << l) - 1));
            return true;
        }
        o.cut += __popcll(cut);
        before += __builtin_amdgcn_readlane(upto, 63);
        slots += __builtin_amdgcn_readlane(kept_upto, 63);
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
        if (high)
            return join(nibble_high(w0, mant), nibble_high(w0 >> 8, mant), nibble_high(w1, mant), nibble_high(w1 >> 8, mant));
        return join(nibble_low(w0, mant), nibble_low(w0 >> 8, mant), nibble_low(w1, mant), nibble_low(w1 >> 8, mant));
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
// Exponent fields of the largest and the smallest number of a set, the latter as 255 less itself: halves of a dword, so that
// one maximum serves for both.  0: no number.
__device__ __forceinline__ uint32_t range_max(uint32_t a, uint32_t b)
{
    typedef uint16_t us2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}
__device__ __forceinline__ uint32_t column_range(uint32_t v)
{
    auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = range_max(p[0], p[1]);
    p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return range_max(p[0], p[1]);
}
// of |v|, if v is finite
__device__ __forceinline__ uint32_t range_of(float v)
{
    const uint32_t e = __float_as_uint(v) >> 23 & 255u;
    return e == 255u ? 0u : e | (255u - e) << 16;
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_range(uint32_t v)
{
    return range_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true));
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
// Exponents that minima are lowered by in their sums of p * minimum, so that minima up to the largest have one over 2^22
// tokens, at p = 2^kSlack all of them; what is lost is 2^-119 a token.
constexpr int kMinDown = 30;
// Exponents between a piece's sum of weights, as it is stored, and 1: results of any size have a sum over 2^12 pieces
constexpr int kSumDown = 20;

// Exponents of the value scales that some row of the item has seen: the largest and the smallest (0 has -127)
struct ValueRange {
    int top = -100, low = 128;
    __device__ __forceinline__ void join(uint32_t range)     // of a whole wave: exponent fields as above
    {
        top = max(top, (int)(range & 0xffffu) - 127);
        low = min(low, 128 - (int)(range >> 16));
    }
};

// 4 dims of a finished row: into y where its item is one piece, else among the pieces' results
template <int D, bool BF16>
__device__ __forceinline__ void put_result(const AttnArgs &a, const Span &t, int pieces, int slot, int kvh, int rows,
                                           int rr, int d, f4 v, float top, float sum)
{
    if (pieces == 1) {
        const int r = t.r0 + rr, i = a.by_group.of(r), h = a.by_group.rest(r);
        const ushort4 w = {round_out<BF16>(v[0]), round_out<BF16>(v[1]), round_out<BF16>(v[2]), round_out<BF16>(v[3])};
        *reinterpret_cast<ushort4 *>(a.y + ((int64_t)(t.s.row0 + i) * a.q_heads + kvh * a.group + h) * D + d) = w;
    } else {
        const int64_t p = ((int64_t)slot * a.kv.heads + kvh) * rows + rr;
        *reinterpret_cast<f4 *>(a.part_o + p * D + d) = v;
        if (d == 0) {
            // sum * 2^top, the sum brought to [2^-kSumDown, 2^(1 - kSumDown))
            const int e = sum > 0.f ? (int)(__float_as_uint(sum) >> 23) - 127 + kSumDown : 0;
            a.part_ml[p] = float2{top + (float)e, ldexpf(sum, -e)};
        }
    }
}

// How a matrix instruction lays things out: COLS = 16 (16x16x32) or 32 (32x32x16) rows of the item are its columns; a lane
// l has column l % COLS and, j being l / COLS, the tokens (64 / QN) * q + 4 j + e of a block, q < QN and e < 4, and as many
// dims of each result.
template <int COLS>
struct Shape;
template <>
struct Shape<16> {
    typedef f4 Acc;
    static constexpr int QN = 4, STEP = 32, TILES = 4, EL = 4;      // STEP: dims (tokens) that an instruction sums over
    static __device__ __forceinline__ f4 mul(h8 a, h8 b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float max_of(float v) { return column_max(v); }
    static __device__ __forceinline__ float sum_of(float v) { return column_sum(v); }
};
template <>
struct Shape<32> {
    typedef float Acc __attribute__((ext_vector_type(16)));
    static constexpr int QN = 8, STEP = 16, TILES = 2, EL = 16;
    static __device__ __forceinline__ Acc mul(h8 a, h8 b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float max_of(float v)
    {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    }
    static __device__ __forceinline__ float sum_of(float v) { return v + __shfl_xor(v, 32); }
};

// COLS * NQ rows of an item as a wave holds them, and what they have summed up so far.
// EVEN: the keys' scales come multiplied by what makes a product of codes and operands an exponent of base 2, for all rows
// alike unless the rows differ too much; else every row has its own factor.
template <int FMT, int D, bool BF16, int COLS, int NQ, bool EVEN>
struct Rows {
    typedef Shape<COLS> S;
    typedef typename S::Acc Acc;
    static constexpr bool I8 = FMT == LOWBIT_KV_I8;
    static constexpr int KS = D / S::STEP, M = D / COLS, EL = S::EL, QN = S::QN, PU = 64 / S::STEP;
    // fp16 results take their weights in two fp16 parts, p = rne(p) + rne(p - rne(p)): one alone costs a result of fp16 as
    // much as its own rounding (4 bits: twice, as codes and minima are summed apart); to one of bf16 it adds 2 %.  The second
    // costs half of the products again: 34 to 36 us for a cache of 146 MB, 140 to 163 us in tiles (64 GFLOP, a window).
    static constexpr int PARTS = BF16 ? 1 : 2;
    typedef Codes<FMT, D> C;
    h8 qf[NQ][KS];
    float c[NQ], qsum[NQ];               // the row's factor of the scales; the sum of its operands
    bool alike;                          // EVEN: all factors are 1
    int see_lo[NQ], see_hi[NQ];          // tokens that the row sees
    Acc o[NQ][M];                        // sum p * vscale * 2^(kTop - E) * code, EL dims of the lane's column
    float mc[NQ], limit[NQ];             // exponent that the row's terms are taken to, and what they may pass it by
    float l[NQ], bias[NQ];               // sums of the lane's p, and of p * vmin * 2^-kMinDown
    int E;
    // Where the item's value scales spread by more than this, the row's own tokens may have small ones, or those that count
    // for much: its sums are then taken to the largest p * vscale so far, by 2^k more than to E.  Up to here the largest
    // operand is at least 2^(kTop - SPREAD), 2^23 (bf16 results: 2^17) times what fp16 rounds next to zero.  A row's own
    // exponents take a maximum and two steps more for each operand: a prompt 656 us for 595, a window 170 for 161, decode 116.4
    // for 116.1, so they are not taken where scales are alike.
    static constexpr int SPREAD = BF16 ? 14 : 8;
    static constexpr int NONE = 1 << 20; // k of a row that has no sums yet
    bool spread;
    int k[NQ];

    // first of the 8 dims that lanes j have in step k
    static __device__ __forceinline__ int dims(int k, int j)
    {
        return COLS == 16 ? k / 2 * 64 + 16 * j + k % 2 * 8 : 16 * k + 8 * j;
    }
    __device__ __forceinline__ void scale_sums(int x, float f)
    {
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int e = 0; e < EL; ++e) o[x][i][e] *= f;
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int e = 0; e < EL; ++e) o[x][i][e] = 0.f;
    }

    // Rows r0 .. of the item, nr of them there.  Returns what the scales of all rows are to be multiplied by (EVEN); the
    // rows of bf16 of all waves then need `meet`, which gives a value's largest and smallest over the workgroup.
    template <typename F>
    __device__ __forceinline__ float load(const AttnArgs &a, const KvSeq &seq, int kvh, int r0, int nr, int lane, F meet)
    {
        const int j = lane / COLS, n = lane % COLS;
        us8 raw[NQ][KS];
        int top[NQ];                     // largest |q| of the row, its bits; 0 where there is none or no number
        // infinite only where a scale of over 2^127 has become so; and as many exponents as it can be lowered by within binary32
        float all = fminf(a.scale2, FLT_MAX);
        const int most = (int)(__float_as_uint(all) >> 23) - 127 + 125;
        alike = true;
        E = ValueRange().top;
        spread = false;
        clear();
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int r = r0 + (x * COLS + n < nr ? x * COLS + n : 0), i = a.by_group.of(r), h = a.by_group.rest(r);
            const uint16_t *src = a.q + (int64_t)(seq.row0 + i) * a.q_stride + (kvh * a.group + h) * D;
            see_hi[x] = seq.pos0 + i + 1;
            see_lo[x] = a.window > 0 ? see_hi[x] - min(a.window, max(seq.len, 1)) : 0;
#pragma unroll
            for (int k = 0; k < KS; ++k) raw[x][k] = *reinterpret_cast<const us8 *>(src + dims(k, j));
            c[x] = EVEN ? 1.f : all;
            qsum[x] = l[x] = bias[x] = mc[x] = 0.f;
            k[x] = 0;
            limit[x] = -INFINITY;
            if constexpr (BF16) {
                top[x] = 0;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) top[x] = max(top[x], raw[x][k][e] & 0x7fff);
                if (COLS == 16) top[x] = max(top[x], __shfl_xor(top[x], 16));
                top[x] = max(top[x], __shfl_xor(top[x], 32));
                if (top[x] >= 0x7f80) top[x] = 0;
            }
        }
        if constexpr (BF16) {
            // into fp16 after a power of two that brings the largest value of the row, or of all rows if none's is smaller
            // by more than 2^8, to [2^14, 2^15), or as near to it as leaves the factor of its scores a normal number: 2^-25
            // of fp16 are less than 2^-14 of a score then, whatever the keys
            int shift_all = 0;
            if constexpr (EVEN) {
                int hi = 0, lo = 0x7fff;
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    hi = max(hi, top[x]);
                    lo = top[x] > 0 ? min(lo, top[x]) : lo;
                }
                meet(hi, lo);
                alike = lo >= hi || (hi >> 7) - (lo >> 7) <= 8;
                shift_all = hi > 0 ? min(141 - (hi >> 7), most) : 0;
                if (alike) all = ldexpf(all, -shift_all);
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const int own = top[x] > 0 ? min(141 - (top[x] >> 7), most) : 0, shift = EVEN && alike ? shift_all : own;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        qf[x][k][e] = (_Float16)ldexpf(__uint_as_float((uint32_t)raw[x][k][e] << 16), shift);
                if (!EVEN || !alike) c[x] = ldexpf(c[x], -own);
            }
        } else {
#pragma unroll
            for (int x = 0; x < NQ; ++x)
#pragma unroll
                for (int k = 0; k < KS; ++k) qf[x][k] = __builtin_bit_cast(h8, raw[x][k]);
        }
        // a query that is not finite makes NaN of its row (q * 0 + q): scores of minus infinity are not told from hidden ones
        const h8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int k = 0; k < KS; ++k) qf[x][k] = __builtin_elementwise_fma(qf[x][k], zero, qf[x][k]);
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            c[x] = fminf(c[x], FLT_MAX);
            if constexpr (!I8) {
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) qsum[x] += (float)qf[x][k][e];
                qsum[x] = S::sum_of(qsum[x]);
            }
        }
        return fminf(all, FLT_MAX);
    }

    // takes the sums to the exponents of the value scales as they are now: what they are to be multiplied by goes to `down`;
    // returns whether that may be other than 1
    __device__ __forceinline__ bool move_to(const ValueRange &range, float (&down)[NQ])
    {
        if (!spread && range.top - range.low > SPREAD) {
            spread = true;
#pragma unroll
            for (int x = 0; x < NQ; ++x) k[x] = limit[x] == -INFINITY ? NONE : 0;
        }
        const int by = range.top - E;
        const float f = spread ? 1.f : ldexpf(1.f, -by);
        E = range.top;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            k[x] = spread ? min(k[x] + by, NONE) : 0;
            down[x] = f;
        }
        return spread | (by != 0);
    }
    // what a sum is to be multiplied by, as an exponent
    __device__ __forceinline__ int unit(int x) const { return E - kTop - k[x]; }

    // acc: products of the queries with a block's codes; leaves the operand of the product with its values.  kl, vl (4
    // bits): minima + 8 scales (the keys' with the factor of their scales, the values' times 2^-kMinDown); vs: times
    // 2^(kTop - E).
    // masked: some row does not see all of the block, whose first token is t0, or its page is missing.
    template <typename KS_, typename KL, typename VS, typename VL>
    __device__ __forceinline__ void weigh(Acc (&acc)[NQ][S::TILES], KS_ ks, KL kl, VS vs, VL vl, bool masked, bool paged,
                                          int64_t t0, int j, const ValueRange &range, h8 (&pf)[PARTS][NQ][PU])
    {
        constexpr int T = 64 / QN;       // tokens from one q to the next
        float down[NQ];                  // what the sums so far are multiplied by, once, at the end
        bool move = move_to(range, down);
        auto s = [&](int x, int q, int e) -> float { return acc[x][q * 4 / EL][q * 4 % EL + e]; };
        auto put = [&](int x, int q, int e, float v) { acc[x][q * 4 / EL][q * 4 % EL + e] = v; };
        // exponents, less the one that the row's terms are taken to
        if (EVEN && alike) {
#pragma unroll
            for (int q = 0; q < QN; ++q) {
                const f4 kq = ks(q), lq = I8 ? f4{} : kl(q);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        put(x, q, e, __builtin_fmaf(s(x, q, e), kq[e],
                                                    I8 ? -mc[x] : __builtin_fmaf(lq[e], qsum[x], -mc[x])));
            }
        } else {
#pragma unroll
            for (int q = 0; q < QN; ++q) {
                const f4 kq = ks(q), lq = I8 ? f4{} : kl(q);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        put(x, q, e, __builtin_fmaf(s(x, q, e), kq[e] * c[x],
                                                    I8 ? -mc[x] : __builtin_fmaf(lq[e] * c[x], qsum[x], -mc[x])));
            }
        }
        // tokens of the block that the lane's rows see, from its own first
        int lo[NQ], hi[NQ];
        if (masked)
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                lo[x] = (int)min(max((int64_t)see_lo[x] - t0, (int64_t)0), (int64_t)kTile) - 4 * j;
                hi[x] = (paged ? (int)min(max((int64_t)see_hi[x] - t0, (int64_t)0), (int64_t)kTile) : 0) - 4 * j;
#pragma unroll
                for (int q = 0; q < QN; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) put(x, q, e, inside(T * q + e, lo[x], hi[x]) ? s(x, q, e) : -INFINITY);
            }
        float top[NQ];
        bool far = false;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float t[QN];
#pragma unroll
            for (int q = 0; q < QN; ++q) t[q] = fmaxf(fmaxf(s(x, q, 0), s(x, q, 1)), fmaxf(s(x, q, 2), s(x, q, 3)));
            top[x] = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
            if (QN == 8) top[x] = fmaxf(top[x], fmaxf(fmaxf(t[QN - 4], t[QN - 3]), fmaxf(t[QN - 2], t[QN - 1])));
            far |= top[x] > limit[x];
        }
        // the exponent moves where a row's first token is seen, and where one has passed it by more than the slack
        if (__any(far)) {
            move = true;
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const float t = S::max_of(top[x]);
                // a whole number, so that what was summed up is taken to it exactly
                const bool none = limit[x] == -INFINITY;
                const float to = t == -INFINITY ? mc[x] : mc[x] + (none ? floorf(t) : fmaxf(floorf(t), 0.f));
                const float by = to - mc[x], alpha = none ? 0.f : exp2_fast(-by);
                mc[x] = to;
                limit[x] = t == -INFINITY ? limit[x] : kSlack;
                l[x] *= alpha;
                bias[x] *= alpha;
                down[x] *= spread ? 1.f : alpha;
                k[x] = spread ? min(k[x] + (int)fminf(by, (float)NONE), NONE) : 0;
#pragma unroll
                for (int q = 0; q < QN; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) put(x, q, e, s(x, q, e) - by);
            }
        }
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int q = 0; q < QN; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = exp2_fast(s(x, q, e));
                    put(x, q, e, p);
                    sum[e % 2] += p;
                }
            l[x] += sum[0] + sum[1];
        }
        // a token that is not seen has p = 0, and counts for nothing even where its scale is no number
        if (masked) {
#pragma unroll
            for (int q = 0; q < QN; ++q) {
                const f4 vq = vs(q), lq = I8 ? f4{} : vl(q);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const bool seen = inside(T * q + e, lo[x], hi[x]);
                        if constexpr (!I8) bias[x] += seen ? s(x, q, e) * lq[e] : 0.f;
                        put(x, q, e, seen ? s(x, q, e) * vq[e] : 0.f);
                    }
            }
        } else {
#pragma unroll
            for (int q = 0; q < QN; ++q) {
                const f4 vq = vs(q), lq = I8 ? f4{} : vl(q);
#pragma unroll
                for (int x = 0; x < NQ; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (!I8) bias[x] = __builtin_fmaf(s(x, q, e), lq[e], bias[x]);
                        put(x, q, e, s(x, q, e) * vq[e]);
                    }
            }
        }
        if (spread)
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                float t = 0.f;
#pragma unroll
                for (int q = 0; q < QN; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) t = fmaxf(t, fabsf(s(x, q, e)));
                t = S::max_of(t);
                const int at = (int)(__float_as_uint(t) >> 23) - 127;
                const int to = t > 0.f && t <= FLT_MAX && at + k[x] > 14 ? min(max(kTop - at, 0), E + 100) : k[x];
                down[x] *= ldexpf(1.f, to - k[x]);
                k[x] = to;
#pragma unroll
                for (int q = 0; q < QN; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) put(x, q, e, ldexpf(s(x, q, e), k[x]));
            }
        if (move)
#pragma unroll
            for (int x = 0; x < NQ; ++x) scale_sums(x, down[x]);
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int u = 0; u < PU; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p = s(x, 2 * u + e / 4, C::order(e % 4));
                    pf[0][x][u][e] = (_Float16)p;
                    if constexpr (PARTS == 2) pf[1][x][u][e] = (_Float16)(p - (float)pf[0][x][u][e]);
                }
    }
};

// Few rows: a workgroup of 4 waves has the 16 * NQ rows of an item, and each wave every 4th block of tokens of its piece.  A
// block's loads are under way while the one before is worked on: its keys are asked for as soon as the last product with the
// keys before them has begun, scales and values likewise, so that they need no registers of their own.
//
// Bound by bytes where many workgroups are resident (decode, 8 bits, 562 MB: 108 us), by a wave's own instructions where few
// are: a block is some 800 of them, 4000 clocks, whatever the number of waves beside it (one sequence of 777 tokens, 8
// heads: 11.4 us; before value scales had their range taken, 11.0 with 4 waves, 11.7 with 8; of 500 tokens 8.3 and 9.3).
template <int FMT, int D, bool BF16, int NQ>
__global__ __launch_bounds__(256, D * NQ > 128 ? 1 : 2) void kv_attention_kernel(AttnArgs a)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    constexpr int W = 4, ROWS = 16 * NQ, KS = D / 32, M = D / 16, DH = D < 128 ? D : 128, LD = DH + 4;
    constexpr int PARTS = Rows<FMT, D, BF16, 16, NQ, false>::PARTS;
    typedef Codes<FMT, D> C;
    __shared__ __attribute__((aligned(16))) float o_s[W * 16 * LD];
    __shared__ float m_s[NQ][W][16], l_s[NQ][W][16], b_s[NQ][W][16];
    __shared__ int e_s[NQ][W][16];
    __shared__ float g_s[NQ][W][16], add_s[NQ][16], top_s[NQ][16], sum_s[NQ][16];

    const int kvh = a.by_heads.rest(blockIdx.x), number = a.by_heads.of(blockIdx.x);
    // whole items: the last tiles of a sequence, its longest, first
    Piece pc = {a.share > 0 ? 0 : a.kv.count * a.tiles - 1 - number, 0, 1, 0, 0, 0, 0};
    if (a.share > 0) {
        const bool found = find_piece(a, ROWS, number, pc);
        if (number == 0 && kvh == 0 && threadIdx.x == 0) a.cuts[0] = int4{pc.cuts, 0, 0, 0};
        if (!found) return;
        if (pc.count > 1 && pc.piece == 0 && kvh == 0 && threadIdx.x == 0)
            a.cuts[1 + pc.cut] = int4{pc.item, pc.slot, pc.count, 0};
    }
    const int item = __builtin_amdgcn_readfirstlane(pc.item), b = a.by_tiles.of(item);
    const Span t = attn_span(a, b, a.by_tiles.rest(item), ROWS);
    if (t.nr <= 0) return;
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
    Rows<FMT, D, BF16, 16, NQ, false> w;
    w.load(a, t.s, kvh, t.r0, t.nr, lane, [](int &, int &) {});

    const int page_size = 1 << a.kv.page_shift;
    BlockRegs<FMT, D> r;
    int blk = begin + wave, page = __builtin_amdgcn_readlane(pages, 0);
    // a block without a page is read from page 0 and not seen
    auto part_of = [&](int p) { return buffer_rsrc(kv_part(a.kv, max(p, 0), kvh), a.kv.part); };
    uint32_t mant = 0x64006400u;
    asm("" : "+v"(mant));
    ValueRange values;

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
                    r.vl[q][e] = ldexpf(__builtin_fmaf(8.f, r.vs[q][e], r.vl[q][e]), -kMinDown);
                }
        }
        const int64_t t0 = (int64_t)blk * kTile;
        // some row does not see all of the block
        const bool masked = page < 0 || blk < (t.seen_lo + kTile - 1) / kTile || blk >= t.seen_hi / kTile;
        // value scales: their range, by their bits, as numbers of either sign and those that are not finite lie above all others
        uint32_t v_top = 0, v_low = ~0u;
        if (masked) {
            // tokens that no row sees: their scales do not count
            const int lo = (int)max((int64_t)0, t.lo - t0), hi = page < 0 ? 0 : (int)min((int64_t)kTile, t.hi - t0);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool seen = inside(16 * q + 4 * j + e, lo, hi);
                    v_low = min(v_low, seen ? __float_as_uint(r.vs[q][e]) : ~0u);
                    r.vs[q][e] = seen ? r.vs[q][e] : 0.f;
                }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) v_low = min(v_low, __float_as_uint(r.vs[q][e]));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) v_top = max(v_top, __float_as_uint(r.vs[q][e]));
        uint32_t range = __builtin_amdgcn_readfirstlane(column_range(v_top >> 23 | (255u - min(v_low >> 23, 255u)) << 16));
        if ((range & 0xffffu) >= 255u) {
            // one by one; those that no row sees are 0 by now, and make a wide range of it
            range = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) range = range_max(range, range_of(r.vs[q][e]));
            range = __builtin_amdgcn_readfirstlane(column_range(range));
        }
        values.join(range);
        const float norm = ldexpf(1.f, kTop - values.top);
#pragma unroll
        for (int q = 0; q < 4; ++q) r.vs[q] *= norm;
        h8 pf[PARTS][NQ][2];
        auto of = [](const f4 *v) { return [v](int q) { return v[q]; }; };
        w.weigh(s, of(r.ks), of(r.kl), of(r.vs), of(r.vl), masked, page >= 0, t0, j, values,
                pf);
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
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
                        w.o[x][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[part][x][u], w.o[x][i], 0, 0, 0);
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

    // the waves' results joined: what each counts for in a row, then 16 rows and up to 128 dims at a time.  One that saw
    // nothing has sums of 0; one whose weight is 0 beside the others' still makes NaN of a row that sees NaN there
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        w.l[x] = column_sum(w.l[x]);
        w.bias[x] = column_sum(w.bias[x]);
        if (j == 0) {
            m_s[x][wave][n] = w.mc[x];
            l_s[x][wave][n] = w.l[x];
            b_s[x][wave][n] = w.bias[x];
            e_s[x][wave][n] = w.unit(x);
        }
    }
    __syncthreads();
    if (threadIdx.x < ROWS) {
        const int x = threadIdx.x / 16, row = threadIdx.x % 16;
        float top = -INFINITY, sum = 0.f, add = 0.f, f[W];
#pragma unroll
        for (int q = 0; q < W; ++q) top = l_s[x][q][row] == 0.f ? top : fmaxf(top, m_s[x][q][row]);
#pragma unroll
        for (int q = 0; q < W; ++q) {
            f[q] = l_s[x][q][row] == 0.f ? 0.f : exp2_fast(m_s[x][q][row] - top);
            sum += f[q] * l_s[x][q][row];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int q = 0; q < W; ++q) {
            add += ldexpf(b_s[x][q][row] * (f[q] * inv), kMinDown);
            g_s[x][q][row] = ldexpf(f[q] * inv, e_s[x][q][row]);
        }
        add_s[x][row] = add;
        top_s[x][row] = top;
        sum_s[x][row] = sum;
    }
#pragma unroll
    for (int x = 0; x < NQ; ++x)
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += DH) {
            if (x > 0 || d0 > 0) __syncthreads();
#pragma unroll
            for (int i = 0; i < DH / 16; ++i)
                *reinterpret_cast<f4 *>(o_s + (wave * 16 + n) * LD + 16 * i + 4 * j) = w.o[x][d0 / 16 + i];
            __syncthreads();
            for (int at = threadIdx.x; at < min(t.nr - 16 * x, 16) * (DH / 4); at += W * 64) {
                const int row = at / (DH / 4), d = at % (DH / 4) * 4;
                const float add = add_s[x][row];
                f4 v = {add, add, add, add};
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    const float g = g_s[x][q][row];
                    const f4 ow = *reinterpret_cast<const f4 *>(o_s + (q * 16 + row) * LD + d);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(ow[e], g, v[e]);
                }
                put_result<D, BF16>(a, t, pc.count, pc.slot + pc.piece, kvh, ROWS, 16 * x + row, d0 + d, v, top_s[x][row],
                                    sum_s[x][row]);
            }
        }
}

// Many rows: a workgroup has kTileRows rows of an item, COLS in each of its W waves, and takes the blocks of its piece one by
// one.  Codes become fp16 operands once for all waves and lie in LDS in the order in which a wave reads them, 16 bytes a lane:
// no permutation, and no bank conflicts.  The 8-byte stores of values for 32x32x16 meet half of the banks twice: 15.8e6 cycles in
// a prompt of 15.8e6 products.
//
// A block is two phases of a wave: M, the products (of the values of the block before, and of the block's keys) with the
// unpacking of what comes next between them, and S, the softmax.  One barrier a block stands between the two: what M(i)
// writes (keys of block i + 1, values of block i) is read in M(i + 1), one barrier later, and lies where M(i - 1) read last,
// one barrier earlier.  Scales of block i + 1 go along with its keys and are read in S(i + 1) by waves that may be one block
// apart: they take turns in four places.
//
// Dims up to 128: 4 waves of 32 rows on 32x32x16, which reads half as much LDS a product as 16x16x32, and two workgroups a
// compute unit, whose phases fall beside each other by themselves.  Against that, 8 waves of 16 rows of which four run a
// phase behind the others by barriers were no faster at any case.  Dims of 256 fill the LDS with one workgroup: 8 waves of 16
// rows (a chunk of 1024 tokens over 4096, 4 heads: 72 us; 4 waves of 32 rows, one on each SIMD: 89).
template <int FMT, int D, bool BF16, int COLS, int W>
__global__ __launch_bounds__(W * 64, W == 8 || D < 256 ? 2 : 1) void kv_attention_tile_kernel(AttnArgs a)
{
    typedef Rows<FMT, D, BF16, COLS, 1, true> R;
    typedef typename R::S Sh;
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    constexpr int ROWS = COLS * W, KS = R::KS, M = R::M, PU = R::PU, QN = R::QN, A = I8 ? 1 : 2;
    typedef Codes<FMT, D> C;
    constexpr int MINE = (C::N + W - 1) / W;                      // KiB of codes of keys (and of values) that a wave unpacks
    constexpr int FRAGS = Sh::TILES * KS;                         // operands of a block's keys (and of its values), 1 KiB each
    static_assert(FRAGS == M * PU, "as many operands of keys as of values");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    h8 *kfrag = reinterpret_cast<h8 *>(lds), *vfrag = kfrag + 2 * FRAGS * 64;   // [2][FRAGS][64] each
    float *arrays = reinterpret_cast<float *>(vfrag + 2 * FRAGS * 64);          // [4][K, V][scale, minimum][64]

    const int kvh = a.by_heads.rest(blockIdx.x), number = a.by_heads.of(blockIdx.x);
    // whole items: the last tiles of a sequence, its longest, first
    Piece pc = {a.share > 0 ? 0 : a.kv.count * a.tiles - 1 - number, 0, 1, 0, 0, 0, 0};
    if (a.share > 0) {
        const bool found = find_piece(a, ROWS, number, pc);
        if (number == 0 && kvh == 0 && threadIdx.x == 0) a.cuts[0] = int4{pc.cuts, 0, 0, 0};
        if (!found) return;
        if (pc.count > 1 && pc.piece == 0 && kvh == 0 && threadIdx.x == 0)
            a.cuts[1 + pc.cut] = int4{pc.item, pc.slot, pc.count, 0};
    }
    const int item = __builtin_amdgcn_readfirstlane(pc.item), b = a.by_tiles.of(item);
    const Span t = attn_span(a, b, a.by_tiles.rest(item), ROWS);
    if (t.nr <= 0) return;
    const int begin = __builtin_amdgcn_readfirstlane(t.first + pc.piece * pc.size);
    const int end = __builtin_amdgcn_readfirstlane(pc.count > 1 ? min(begin + pc.size, t.end) : t.end);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane / COLS, n = lane % COLS;
    const int page_size = 1 << a.kv.page_shift;
    // the wave's own rows, and what they see
    const int w0 = wave * COLS, wn = min(t.nr - w0, COLS);
    const Span ws = attn_rows(a, t.s, t.r0 + w0, wn);

    auto pages_of = [&](int blk) { return blk + lane < end ? kv_page(a.kv, b, blk + lane) : -1; };
    int pages = pages_of(begin);
    R w;
    const float k_factor = w.load(a, t.s, kvh, wn > 0 ? t.r0 + w0 : t.r0, wn, lane, [&](int &hi, int &lo) {
        int *m = reinterpret_cast<int *>(lds);
        for (int o = 32; o > 0; o >>= 1) {
            hi = max(hi, __shfl_xor(hi, o));
            lo = min(lo, __shfl_xor(lo, o));
        }
        if (lane == 0) {
            m[wave] = hi;
            m[W + wave] = lo;
        }
        __syncthreads();
        for (int q = 0; q < W; ++q) {
            hi = max(hi, m[q]);
            lo = min(lo, m[W + q]);
        }
        hi = __builtin_amdgcn_readfirstlane(hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        __syncthreads();
    });
    uint32_t mant = 0x64006400u;
    asm("" : "+v"(mant));

    // Codes on their way to LDS: keys of a block, values of the one before.  Past the last block its loads are repeated, so
    // that nothing in phase M hangs on a branch.
    u4 kraw[MINE], vraw[MINE];
    int page_k = -1;                     // page of the keys in kraw
    auto part_of = [&](int page) { return buffer_rsrc(kv_part(a.kv, max(page, 0), kvh), a.kv.part); };
    auto in_page = [&](int blk) { return (blk * kTile) & (page_size - 1); };
    auto fetch = [&](int blk) {          // the keys of blk, the values of the block before
        const int i = blk - begin, page_v = page_k;
        if ((i & 63) == 0 && i > 0) pages = pages_of(blk);
        page_k = blk < end ? __builtin_amdgcn_readlane(pages, i & 63) : page_k;
        const auto pk = part_of(page_k), pv = part_of(page_v);
        const int at_k = kv_code_bytes(FMT, in_page(min(blk, end - 1)), D);
        const int at_v = kv_code_bytes(FMT, page_size + in_page(max(blk - 1, begin)), D);
#pragma unroll
        for (int q = 0; q < MINE; ++q) {
            const int chunk = wave + q * W;
            if (C::N % W != 0 && chunk >= C::N) break;
            kraw[q] = BlockRegs<FMT, D>::get(pk, lane * 16, at_k + chunk * 1024);
            vraw[q] = BlockRegs<FMT, D>::get(pv, lane * 16, at_v + chunk * 1024);
        }
    };
    // The operands that a wave unpacks, one by one: OPS / 2 of the keys of the piece's block i + 1, then as many of the values
    // of block i.  A KiB of codes holds 2 operands of 8 bits, 4 of 4 bits: of keys, two steps of 64 dims (of 16 tokens each);
    // of values, two steps of 32 tokens (of 16 dims each).
    constexpr int PER = I8 ? 2 : 4, OPS = 2 * MINE * PER;
    auto unpack = [&](int op, int i) {
        const int q = op / PER % MINE, v = op % PER, chunk = wave + q * W;
        if (C::N % W != 0 && chunk >= C::N) return;
        // the page's lane: 16 bytes of dims 16 sj of token sr, tokens 4 sj of dim sr
        const int sj = lane >> 4, sr = lane & 15;
        if (op < OPS / 2) {
            const h8 f = C::key_of(kraw[q], v, mant);
            const int d = chunk % (D / 64), q0 = chunk / (D / 64) * (PER / 2) + v / 2;   // 64 dims, 16 tokens
            h8 *to = kfrag + (i + 1 & 1) * FRAGS * 64;
            if constexpr (COLS == 16) to[(q0 * KS + 2 * d + v % 2) * 64 + lane] = f;
            else to[(q0 / 2 * KS + 4 * d + sj) * 64 + v % 2 * 32 + q0 % 2 * 16 + sr] = f;
        } else {
            const h8 f = C::value_of(vraw[q], v / 2, v % 2, mant);
            const int d = chunk * (PER / 2) + v / 2;                                     // 16 dims
            h8 *to = vfrag + (i & 1) * FRAGS * 64;
            if constexpr (COLS == 16) to[(d * 2 + v % 2) * 64 + lane] = f;
            else
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    reinterpret_cast<h4 *>(to + (d / 2 * 4 + v % 2 * 2 + u) * 64 + sj % 2 * 32 + d % 2 * 16 + sr)[sj / 2] =
                        h4{f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]};
        }
    };
    // Scales of a block on their way to LDS, a token a lane.  Every wave has all of them: the range of the value scales so far
    // (of tokens that some row sees, infinities and NaN aside) is the same in each, and comes about in steps that fit between
    // products.
    float scale[2], low[2];
    uint32_t v_range;
    ValueRange values;
    int page_a = -1;
    auto fetch_scales = [&](int blk) {   // of blk, whose page is page_k
        page_a = page_k;
        const auto part = part_of(page_k);
        const int from = 2 * kv_code_bytes(FMT, page_size, D) + in_page(min(blk, end - 1)) * 4;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            scale[v] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part, lane * 4, from + v * A * page_size * 4, 0));
            if constexpr (!I8)
                low[v] = __uint_as_float(
                    __builtin_amdgcn_raw_buffer_load_b32(part, lane * 4, from + (v * A + 1) * page_size * 4, 0));
        }
    };
    constexpr int kScaleSteps = 8;
    auto unpack_scales = [&](int step, int i) {
        if (step == 0) {
            const int64_t token = (int64_t)(begin + i) * kTile + lane;
            v_range = ((token >= t.lo) & (token < t.hi) & (page_a >= 0)) ? range_of(scale[1]) : 0u;
        }
        if (step == 1) v_range = dpp_range<0xb1>(v_range);
        if (step == 2) v_range = dpp_range<0x4e>(v_range);
        if (step == 3) v_range = dpp_range<0x141>(v_range);
        if (step == 4) v_range = dpp_range<0x140>(v_range);
        if (step == 5) v_range = column_range(v_range);
        if (step == 6) values.join(__builtin_amdgcn_readfirstlane(v_range));
        if (step == 7) {
            float *at = arrays + (i & 3) * 2 * A * 64 + lane;
            if (wave == 0) {
                at[0] = scale[0] * k_factor;
                if constexpr (!I8) at[64] = __builtin_fmaf(8.f, scale[0], low[0]) * k_factor;
            }
            if (wave == 1) {
                at[A * 64] = ldexpf(scale[1], kTop - values.top);
                if constexpr (!I8) at[3 * 64] = ldexpf(__builtin_fmaf(8.f, scale[1], low[1]), -kMinDown);
            }
        }
    };

    const int count = end - begin;
    typename R::Acc s[1][Sh::TILES];
    h8 pf[R::PARTS][1][PU];
    auto no_weights = [&] {
#pragma unroll
        for (int part = 0; part < R::PARTS; ++part)
#pragma unroll
            for (int u = 0; u < PU; ++u) pf[part][0][u] = h8{0, 0, 0, 0, 0, 0, 0, 0};
    };
    no_weights();
    // Products of the values of block i - 1, then of the keys of block i; kAhead operands are under way from LDS, and the
    // unpacking goes in between: the matrix cores leave the vector unit three of four of its turns.
    constexpr int kAhead = 6;
    auto multiply = [&](auto keys, int i) {
        constexpr bool KEYS = decltype(keys)::value;
        constexpr int ALL = KEYS ? 2 * FRAGS : FRAGS;
        const h8 *vf = vfrag + (i - 1 & 1) * FRAGS * 64 + lane, *kf = kfrag + (i & 1) * FRAGS * 64 + lane;
        h8 ring[kAhead];
        auto ask = [&](int q) { ring[q % kAhead] = q < FRAGS ? vf[q * 64] : kf[(q - FRAGS) * 64]; };
#pragma unroll
        for (int q = 0; q < kAhead; ++q) ask(q);
#pragma unroll
        for (int q = 0; q < FRAGS; ++q) {
            const h8 f = ring[q % kAhead];
#pragma unroll
            for (int part = 0; part < R::PARTS; ++part) w.o[0][q / PU] = Sh::mul(f, pf[part][0][q % PU], w.o[0][q / PU]);
            if (q + kAhead < ALL) ask(q + kAhead);
            if (KEYS)
#pragma unroll
                for (int op = 0; op < OPS; ++op)
                    if (q == op * FRAGS / OPS) unpack(op, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!KEYS) return;
        fetch(begin + i + 2);
#pragma unroll
        for (int q = 0; q < FRAGS; ++q) {
            const h8 f = ring[(FRAGS + q) % kAhead];
            const int t = q / KS, k = q % KS;
            s[0][t] = Sh::mul(f, w.qf[0][k], k == 0 ? typename R::Acc{} : s[0][t]);
            if (FRAGS + q + kAhead < ALL) ask(FRAGS + q + kAhead);
#pragma unroll
            for (int step = 0; step < kScaleSteps; ++step)
                if (q == step * FRAGS / kScaleSteps) unpack_scales(step, i + 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        fetch_scales(begin + i + 2);
    };
    if (count > 0) {
        fetch(begin);
        int page_next = page_k;          // of block i + 1
        fetch_scales(begin);
#pragma unroll
        for (int op = 0; op < OPS / 2; ++op) unpack(op, -1);
#pragma unroll
        for (int step = 0; step < kScaleSteps; ++step) unpack_scales(step, 0);
        fetch(begin + 1);                // keys of block 1, values of block 0
        fetch_scales(begin + 1);
        __syncthreads();
        for (int i = 0; i < count; ++i) {
            // M
            const int page = page_next, blk = begin + i;
            const ValueRange now = values;
            page_next = page_k;
            __builtin_amdgcn_s_setprio(1);
            multiply(std::true_type{}, i);
            if (i == 0) w.clear();                       // no values were there yet
            // the keys' scales before the barrier, the others as they are needed
            const float *ar = arrays + (i & 3) * 2 * A * 64 + 4 * j;
            auto get = [ar](int which) {
                return [=](int q) { return *reinterpret_cast<const f4 *>(ar + which * 64 + 64 / QN * q); };
            };
            f4 ks[QN];
#pragma unroll
            for (int q = 0; q < QN; ++q) ks[q] = get(0)(q);
            __builtin_amdgcn_s_setprio(0);
            __syncthreads();
            // S
            if (wn > 0 && blk >= ws.first && blk < ws.end && page >= 0) {
                const bool masked = blk < (ws.seen_lo + kTile - 1) / kTile || blk >= ws.seen_hi / kTile;
                w.weigh(s, [&](int q) { return ks[q]; }, get(1), get(A), get(3), masked, true, (int64_t)blk * kTile, j,
                        now, pf);
            } else {
                no_weights();
            }
        }
        multiply(std::false_type{}, count);              // the values of the last block
    }

    const float sum = Sh::sum_of(w.l[0]), low_sum = Sh::sum_of(w.bias[0]);
    if (n >= wn) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum, add = ldexpf(low_sum * inv, kMinDown);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int q = 0; q < R::EL / 4; ++q) {
            f4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = ldexpf(w.o[0][i][4 * q + e] * inv, w.unit(0)) + add;
            put_result<D, BF16>(a, t, pc.count, pc.slot + pc.piece, kvh, ROWS, w0 + n, COLS * i + 8 * q + 4 * j, v, w.mc[0],
                                sum);
        }
}

// The pieces of a cut item's rows joined: each has its own normalised result, and weighs sum * 2^maximum.  The items of both
// launches are joined by one, whose workgroups take `per` rows of an item and head at a time, dim / 4 lanes a row.  Where an
// item has few pieces each row is the work of its own lanes; else rows come one by one, 256 / (dim / 4) pieces at a time.
// 4 to 6 us, most of it the launch and four loads one after the other; 34 MB of pieces of tiles, 13 us.
struct JoinArgs {
    AttnArgs a[2];                       // share = 0: nothing of it is cut
    int rows[2], per[2], groups[2], cuts[2];
    int grid[2];                         // workgroups of each
};
constexpr int kJoinGroups = 2048;        // as many workgroups as are resident at once
constexpr int kFewPieces = 8;

template <int D, bool BF16, bool TILES>
__global__ __launch_bounds__(256, 6) void kv_attention_join_kernel(JoinArgs p)
{
    constexpr int LANES = D / 4, G = 256 / LANES;
    __shared__ f4 part[G][LANES];
    __shared__ float sums[G];
    const int which = TILES && (int)blockIdx.x >= p.grid[0];
    const AttnArgs &a = p.a[which];
    const int heads = a.kv.heads, rows = p.rows[which], per = p.per[which], groups = p.groups[which], grid = p.grid[which];
    const int lane = threadIdx.x & 63, g = threadIdx.x / LANES, d = threadIdx.x % LANES * 4;
    for (int at = blockIdx.x - (which ? p.grid[0] : 0);; at += grid) {
        const int cut = at / heads / groups;
        if (cut >= p.cuts[which]) return;
        const int4 it = a.cuts[1 + cut];             // asked for beside their number
        if (cut >= a.cuts[0].x) return;
        const int kvh = at % heads, r0 = at / heads % groups * per;
        const int item = __builtin_amdgcn_readfirstlane(it.x), pieces = __builtin_amdgcn_readfirstlane(it.z);
        const Span t = attn_span(a, a.by_tiles.of(item), a.by_tiles.rest(item), rows);
        const int64_t step = (int64_t)heads * rows, base = ((int64_t)it.y * heads + kvh) * rows;
        if (TILES && per > 1 && pieces <= kFewPieces) {
            const int rr = r0 + g;
            if (g >= per || rr >= t.nr) continue;
            float2 ml[kFewPieces];
            f4 v = {0.f, 0.f, 0.f, 0.f};
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < kFewPieces; ++i) {
                ml[i] = a.part_ml[base + rr + min(i, pieces - 1) * step];
                if (i >= pieces) ml[i].y = 0.f;
            }
#pragma unroll
            for (int i = 0; i < kFewPieces; ++i) top = ml[i].y != 0.f ? fmaxf(top, ml[i].x) : top;
#pragma unroll
            for (int i0 = 0; i0 < kFewPieces; i0 += 4) {
                if (i0 >= pieces) break;
                f4 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = *reinterpret_cast<const f4 *>(a.part_o + (base + rr + min(i0 + i, pieces - 1) * step) * D + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = ml[i0 + i].y == 0.f ? 0.f : ml[i0 + i].y * exp2_fast(ml[i0 + i].x - top);
                    sum += f;
                    v += i0 + i < pieces ? o[i] * f : f4{0.f, 0.f, 0.f, 0.f};
                }
            }
            put_result<D, BF16>(a, t, 1, 0, kvh, rows, rr, d, v * (sum == 0.f ? 0.f : 1.f / sum), 0.f, 0.f);
            continue;
        }
        for (int rr = r0; rr < min(r0 + per, t.nr); ++rr) {
            float top = -INFINITY;
            for (int i = lane; i < pieces; i += 64) {
                const float2 ml = a.part_ml[base + rr + i * step];
                if (ml.y != 0.f) top = fmaxf(top, ml.x);
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            f4 v = {0.f, 0.f, 0.f, 0.f};
            float sum = 0.f;
#pragma unroll 4
            for (int i = g; i < pieces; i += G) {
                const float2 ml = a.part_ml[base + rr + i * step];
                const f4 o = *reinterpret_cast<const f4 *>(a.part_o + (base + rr + i * step) * D + d);
                const float f = ml.y == 0.f ? 0.f : ml.y * exp2_fast(ml.x - top);
                sum += f;
                v += o * f;
            }
            part[g][threadIdx.x % LANES] = v;
            if (d == 0) sums[g] = sum;
            __syncthreads();
            if (threadIdx.x < LANES) {
                v = f4{0.f, 0.f, 0.f, 0.f};
                sum = 0.f;
#pragma unroll 4
                for (int i = 0; i < G; ++i) {
                    v += part[i][threadIdx.x];
                    sum += sums[i];
                }
                put_result<D, BF16>(a, t, 1, 0, kvh, rows, rr, d, v * (sum == 0.f ? 0.f : 1.f / sum), 0.f, 0.f);
            }
            __syncthreads();                 // the row is read before the next is written
        }
    }
}

constexpr int kTileRows = 128;
// Blocks up to which an item is not worth a second launch: one sequence of 500 tokens, 8 heads of 128, 8 bits, takes 8.3 us
// whole and 11.7 in pieces; of 1800 tokens, 17.0 and 10.8.
constexpr int kWholeBlocks = 16;
// Rows of a sequence up to which it goes with the few, where others have many: 1024 rows beside 31 sequences of one row, 4
// heads of 256, take 118 us so, 178 all in tiles.
constexpr int64_t kFewBeside = 16;
// Rows of a sequence that the kernel for few takes: as many as its registers hold.  A tile does the products of 128 rows
// whatever there are.  8 bits, sequences of up to 4001 tokens: 24 of 40 rows, 2 heads of 64, 21.6 us, 29.2 in tiles (of 64 rows
// 23.8 and 29.9; 4 bits 24.8 and 32.9, of 64 rows 26.9 and 34.0); 16 of 32 rows, 4 heads of 128, 23.6 and 36.4; 16 of 16 rows,
// 4 heads of 256, 26.1 and 39.8.
int64_t few_rows(int dim) { return dim == 64 ? 64 : dim == 128 ? 32 : 16; }
// Workgroups that are resident at once, which the pieces fill: two on a compute unit, one where LDS (tiles of 256 dims) or
// registers (few rows, more than 128 sums a lane) leave room for no more.  Few rows, with the other of 256 and 512: 562 MB
// 114.5 us for 120.5; 40 rows of 64 dims 22.2 for 28.3; tiles of 256 dims 118 for 134.
int resident(int dim, int nq) { return dim * nq > 128 ? 256 : 512; }

// A launch over the sequences of over < rows * group <= upto
struct AttnPlan {
    bool tile;
    int nq, rows;                 // rows of an item: 16 * nq for all waves (few), kTileRows (tile)
    int64_t over, upto, pieces, slots;   // workgroups for each head at most, results of pieces
    int tiles, share, cuts;              // cuts: items that are cut, at most
};
int64_t plan_bytes(const AttnPlan &p, const KvArgs &a)
{
    if (p.share == 0) return 0;
    // 2 * share cut items have a place also where offsets that go back make more items than there are rows for
    return p.slots * a.heads * p.rows * (a.dim * 4 + 8) + (2 * (int64_t)p.share + 1) * (int64_t)sizeof(int4);
}
void cut_plan(AttnPlan &p, const KvArgs &a, int group, int64_t most_rows, int places)
{
    p.tiles = (int)((most_rows + p.rows - 1) / p.rows);
    const int64_t items = (int64_t)p.tiles * a.count, blocks = ((int64_t)a.width << a.page_shift) / kTile;
    const bool cut = items <= kMaxItems && blocks > kWholeBlocks;
    p.share = cut ? std::max(places / a.heads, 1) : 0;
    // tiles that there can be: whole ones of all rows, and a sequence's last
    const int64_t there = std::min(items, (int64_t)a.rows * group / p.rows + std::min(a.count, a.rows));
    // T / size is at most 2 * share, 1.5 * share for tiles, and a cut item's pieces less than twice its part of that; nor are
    // they more than its table's blocks make of kMinPiece each
    const int64_t most = 2 * (int64_t)p.share, least = (blocks + kMinPiece - 1) / kMinPiece;
    p.pieces = cut ? std::min(there + most, items * least) : items;
    p.slots = std::min(p.tile ? 3 * (int64_t)p.share : 2 * most, items * least);
    p.cuts = (int)std::min<int64_t>(there, most);
}
// one launch or two: sequences of many rows first
int attn_plan(const KvArgs &a, int q_heads, AttnPlan *p)
{
    const int group = q_heads / a.heads;
    const int64_t rows = (int64_t)a.max_rows * group, few = few_rows(a.dim);
    int n = 0;
    if (rows > few) {
        AttnPlan &t = p[n++];
        t.tile = true;
        t.nq = 0;
        t.rows = kTileRows;
        t.over = a.count > 1 ? kFewBeside : 0;
        t.upto = INT64_MAX;
        cut_plan(t, a, group, rows, resident(a.dim, 1));
        if (a.count == 1) return n;
    }
    AttnPlan &f = p[n++];
    const int64_t most = rows > few ? kFewBeside : rows;
    f.tile = false;
    f.nq = most <= 16 ? 1 : most <= 32 ? 2 : 4;
    f.rows = 16 * f.nq;
    f.over = 0;
    f.upto = rows > few ? kFewBeside : INT64_MAX;
    cut_plan(f, a, group, most, resident(a.dim, f.nq));
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
    int64_t all = 0;
    for (int i = 0; i < n; ++i) all += plan_bytes(p[i], a);
    return (size_t)all;
}

hipError_t launch_kv_attention(const KvArgs &kv, const void *q, int64_t q_stride, int q_heads, int bf16, float scale,
                               int window, void *y, void *ws, hipStream_t s)
{
    AttnPlan plans[2];
    const int n = attn_plan(kv, q_heads, plans);
    JoinArgs joined{};
    uint8_t *free = static_cast<uint8_t *>(ws);
    auto launch = [&](const AttnPlan &p, auto fmt, auto dim, auto bf) {
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value;
        constexpr bool B = decltype(bf)::value;
        AttnArgs a{kv, static_cast<const uint16_t *>(q), q_stride, q_heads, q_heads / kv.heads, window, scale * kLog2e,
                   static_cast<uint16_t *>(y), Divisor(q_heads / kv.heads), Divisor(p.tiles), Divisor(kv.heads), p.tiles,
                   p.over, p.upto, p.share, p.tile, nullptr, nullptr, nullptr};
        if (p.share > 0) {
            a.part_o = reinterpret_cast<float *>(free);
            a.part_ml = reinterpret_cast<float2 *>(a.part_o + p.slots * kv.heads * p.rows * kv.dim);
            a.cuts = reinterpret_cast<int4 *>(a.part_ml + p.slots * kv.heads * p.rows);
            free += plan_bytes(p, kv);
        }
        const unsigned grid = (unsigned)(p.pieces * kv.heads);
        auto tile = [&](auto cols, auto waves) {
            constexpr int COLS = decltype(cols)::value, W = decltype(waves)::value;
            constexpr size_t lds = 512 * D + (F == LOWBIT_KV_I8 ? 2048 : 4096);
            auto kernel = kv_attention_tile_kernel<F, D, B, COLS, W>;
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
        typedef std::integral_constant<int, 4> four;
        hipError_t e;
        if (p.tile) {
            typedef std::integral_constant<int, 16> c16;
            typedef std::integral_constant<int, 32> c32;
            typedef std::integral_constant<int, 4> w4;
            typedef std::integral_constant<int, 8> w8;
            if constexpr (D == 256) e = tile(c16{}, w8{});
            else e = tile(c32{}, w4{});
        } else {
            auto few = [&](auto nq) {
                constexpr int NQ = decltype(nq)::value;
                kv_attention_kernel<F, D, B, NQ><<<grid, 256, 0, s>>>(a);
                return hipGetLastError();
            };
            if constexpr (D == 64) e = p.nq == 1 ? few(one{}) : p.nq == 2 ? few(two{}) : few(four{});
            else if constexpr (D == 128) e = p.nq == 1 ? few(one{}) : few(two{});
            else e = few(one{});
        }
        const int k = &p == plans ? 0 : 1, most = (int)std::min<int64_t>(p.rows, (int64_t)kv.max_rows * a.group);
        joined.a[k] = a;
        joined.rows[k] = p.rows;
        joined.per[k] = p.tile ? 4 : 1;
        joined.groups[k] = (most + joined.per[k] - 1) / joined.per[k];
        joined.cuts[k] = p.cuts;
        if (p.share > 0) joined.grid[k] = (int)std::min<int64_t>((int64_t)p.cuts * kv.heads * joined.groups[k], kJoinGroups);
        const int grid_all = joined.grid[0] + joined.grid[1];
        if (e != hipSuccess || k + 1 < n || grid_all == 0) return e;
        if (plans[0].tile) kv_attention_join_kernel<D, B, true><<<grid_all, 256, 0, s>>>(joined);
        else kv_attention_join_kernel<D, B, false><<<grid_all, 256, 0, s>>>(joined);
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
