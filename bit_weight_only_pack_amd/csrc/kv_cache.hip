// kv_cache.hip -- rows of keys and values quantised into the pages of a cache,
// and read back from them.
//
// A row is the dim values of one token and head.  8 bits: amax = max |x|, scale
// = amax / 127, code = rne(x * (127 / amax)).  4 bits: lo = min x, h = (max x -
// lo) / 2, scale = h / 7.5, code = rne((x - lo) / 2 * (15 / h)), value = code *
// scale + lo.  Halves, so that no difference of finite values overflows.  Every
// step is one binary32 rounding, so equal rows give equal bytes.
//
// One workgroup takes 64 tokens of one sequence that lie in one block of a page,
// for the keys or the values of one head, and asks for all of its rows at once.
// A wave holds 4 tokens in lanes 16 apart (8 tokens of 64 dims), 8 or 16 dims to
// a lane.  Keys go to memory as they are, 8 (4) bytes a lane.  The page holds
// values by dim, 4 tokens to a dword: four lanes exchange their bytes by swaps of
// lane rows, the dwords meet in LDS in the page's order, and leave it 16 bytes at
// a time where the block is whole, by dwords and bytes at its ends: no byte of
// another token is written.
//
// Both directions are bound by bytes: 16 sequences of up to 8192 tokens read, 8
// bits, 8 heads of 128 dims, move 305 MB in 59 us, 5.2 TB/s, as fast as a large
// copy.  A prompt of 16384 rows, 102 MB, is written in 27 us and read back in 18
// (its pages are still in the last cache then).  32 rows of 32 sequences take 5
// us, the launch and one round of loads and stores.
#include <cfloat>

#include "kv_cache.hpp"

namespace lowbit {

namespace {

constexpr int kThreads = 256;


template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t v)
{
    if constexpr (BF16) return __uint_as_float((uint32_t)v << 16);
    return (float)__builtin_bit_cast(_Float16, v);
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_f32(float v)
{
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// The block of 64 tokens that a workgroup works on
struct Block {
    int head, page, block;               // block of 64 tokens of the sequence, may be negative
    bool values;
    int lo, hi;                          // tokens of the block that rows stand for
    int64_t row;                         // row of the block's token 0 (may name none)
};
__device__ __forceinline__ bool kv_block(const KvArgs &a, int blocks, Block &o)
{
    int id = blockIdx.x;
    const int hv = id % (2 * a.heads);
    id /= 2 * a.heads;
    const int b = id / blocks;
    const KvSeq s = kv_sequence(a, b);
    o.head = hv % a.heads;
    o.values = hv >= a.heads;
    o.block = (s.pos0 >> 6) + id % blocks;
    const int64_t base = (int64_t)o.block * 64;
    o.lo = (int)max((int64_t)0, s.pos0 - base);
    o.hi = (int)min((int64_t)64, (int64_t)s.pos0 + s.n - base);
    o.row = s.row0 + base - s.pos0;
    if (o.lo >= o.hi) return false;
    o.page = kv_page(a, b, o.block);
    return true;
}

// Byte of (token t, first dim d of 8) in a page's keys
template <int FMT, int D>
__device__ __forceinline__ int key_byte(int t, int d)
{
    if (FMT == LOWBIT_KV_I8) return ((t / 16 * (D / 64) + d / 64) * 4 + d % 64 / 16) * 256 + t % 16 * 16 + d % 16;
    return ((t / 32 * (D / 64) + d / 64) * 4 + d % 64 / 16) * 256 + t % 16 * 16 + t % 32 / 16 * 8 + d % 16 / 8 * 4;
}
// Dword of a block of values in LDS: 4 tokens from 4 * quad on, byte b of a token's row (4 bits: 16 of every 32 dims).
// The page's order but for the last two bits, which are turned by b / 16 so that 64 lanes meet few banks twice.
__device__ __forceinline__ int value_word(int quad, int b)
{
    return (b / 16 * 4 + quad % 4) * 64 + b % 16 * 4 + (quad / 4 ^ (b / 16 & 3));
}

template <int LANES, typename T, typename F>
__device__ __forceinline__ T across(T v, F f)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = f(v, (T)__shfl_xor(v, o));
    return v;
}

// Four tokens in lanes l, l + 16, l + 32, l + 48, with 8 bytes each (a: 0..3, b: 4..7), become 4 tokens of bytes 2 r and
// 2 r + 1 in the lanes of row r (a, b).  The inverse is turn_back.
__device__ __forceinline__ void turn(uint32_t &a, uint32_t &b)
{
    const auto p = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    const uint32_t x = __builtin_amdgcn_perm(p[1], p[0], 0x05040100u), y = __builtin_amdgcn_perm(p[1], p[0], 0x07060302u);
    const auto q = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    a = __builtin_amdgcn_perm(q[1], q[0], 0x06020400u);
    b = __builtin_amdgcn_perm(q[1], q[0], 0x07030501u);
}
__device__ __forceinline__ void turn_back(uint32_t &a, uint32_t &b)
{
    const uint32_t x = __builtin_amdgcn_perm(b, a, 0x06020400u), y = __builtin_amdgcn_perm(b, a, 0x07030501u);
    const auto q = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    const uint32_t c = __builtin_amdgcn_perm(q[1], q[0], 0x05040100u), d = __builtin_amdgcn_perm(q[1], q[0], 0x07060302u);
    const auto p = __builtin_amdgcn_permlane32_swap(c, d, false, false);
    a = p[0];
    b = p[1];
}

// How a workgroup shares out a block: ROUNDS times, a wave takes QUADS times 4 tokens, a lane CH times 8 dims of one.
template <int D>
struct Share {
    static constexpr int LANES = D < 128 ? D / 8 : 16, CH = D / (8 * LANES), QUADS = 16 / LANES;
    static constexpr int ROUNDS = 16 / (kThreads / 64 * QUADS);
    int l, t4, wave, first;              // lane of its row, token of its quad; first quad of the block that has rows
    __device__ __forceinline__ explicit Share(const Block &o)
    {
        const int lane = threadIdx.x & 63;
        l = lane % LANES;
        t4 = lane / 16;
        wave = threadIdx.x / 64;
        first = o.lo / 4 + lane / LANES % QUADS;
    }
    __device__ __forceinline__ int quad(int round) const { return first + (round * (kThreads / 64) + wave) * QUADS; }
    __device__ __forceinline__ int dim(int ch) const { return ch * 128 + l * 8; }
};

template <int FMT, int D, bool BF16, bool PASSING>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvArgs a, const uint16_t *k, int64_t k_stride,
                                                            const uint16_t *v, int64_t v_stride, int blocks)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    typedef Share<D> S;
    constexpr int IMAGE = kv_code_bytes(FMT, 64, D);
    __shared__ __attribute__((aligned(16))) uint32_t image[IMAGE / 4];
    Block o;
    if (!kv_block(a, blocks, o)) return;
    const S sh(o);
    const uint16_t *src = o.values ? v : k;
    const int64_t stride = o.values ? v_stride : k_stride;
    us8 raw[S::ROUNDS][S::CH];
#pragma unroll
    for (int i = 0; i < S::ROUNDS; ++i) {
        const int t = sh.quad(i) * 4 + sh.t4;
#pragma unroll
        for (int c = 0; c < S::CH; ++c) {
            raw[i][c] = us8{0, 0, 0, 0, 0, 0, 0, 0};
            if (t >= o.lo && t < o.hi) {
                const us8 *at = reinterpret_cast<const us8 *>(src + (o.row + t) * stride + o.head * D + sh.dim(c));
                raw[i][c] = PASSING ? __builtin_nontemporal_load(at) : *at;
            }
        }
    }
    if (o.page < 0) return;
    const int page_size = 1 << a.page_shift, in_page = (o.block * 64) & (page_size - 1);
    uint8_t *part = kv_part(a, o.page, o.head);
    const int codes = kv_code_bytes(FMT, page_size, D);
    float *arrays = reinterpret_cast<float *>(part + 2 * codes) + (o.values ? kv_arrays(FMT) / 2 * page_size : 0);

#pragma unroll
    for (int i = 0; i < S::ROUNDS; ++i) {
        const int quad = sh.quad(i), t = quad * 4 + sh.t4;
        const bool have = t >= o.lo && t < o.hi;
        if (!__any(have)) break;
        float x[S::CH][8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < S::CH; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[c][e] = to_f32<BF16>(raw[i][c][e]);
                top = max(top, __float_as_uint(x[c][e]) & 0x7fffffffu);
            }
        top = across<S::LANES>(top, [](uint32_t p, uint32_t q) { return max(p, q); });
        const bool bad = top >= 0x7f800000u;         // an infinity or a NaN
        float scale, low = 0.f;
        uint32_t w[S::CH][2];                        // 8 bits: codes in bytes; 4 bits: the same before they are packed
        if constexpr (I8) {
            const float amax = __uint_as_float(top), inv = fminf(127.f / amax, FLT_MAX);
            scale = amax / 127.f;
#pragma unroll
            for (int c = 0; c < S::CH; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w[c][h] = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[c][h] |= (bad ? 128u : (uint32_t)((int)rintf(x[c][4 * h + e] * inv) + 128)) << (8 * e);
                }
        } else {
            float lo = x[0][0], hi = x[0][0];
#pragma unroll
            for (int c = 0; c < S::CH; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    lo = fminf(lo, x[c][e]);
                    hi = fmaxf(hi, x[c][e]);
                }
            lo = across<S::LANES>(lo, [](float p, float q) { return fminf(p, q); });
            hi = across<S::LANES>(hi, [](float p, float q) { return fmaxf(p, q); });
            const float h = 0.5f * hi - 0.5f * lo, inv = fminf(15.f / h, FLT_MAX);
            scale = h / 7.5f;
            low = bad ? 0.f : lo;
#pragma unroll
            for (int c = 0; c < S::CH; ++c)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    w[c][g] = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[c][g] |= (bad ? 0u : (uint32_t)(int)rintf((0.5f * x[c][4 * g + e] - 0.5f * lo) * inv)) << (8 * e);
                }
        }
        if (have && sh.l == 0) {
            arrays[in_page + t] = bad ? __uint_as_float(0x7fc00000u) : scale;
            if constexpr (!I8) arrays[page_size + in_page + t] = low;
        }
#pragma unroll
        for (int c = 0; c < S::CH; ++c) {
            if (!o.values) {
                uint8_t *to = part + key_byte<FMT, D>(in_page + t, sh.dim(c));
                if constexpr (I8) {
                    if (have) *reinterpret_cast<uint2 *>(to) = uint2{w[c][0], w[c][1]};
                } else {
                    uint32_t n = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) n |= (w[c][e / 4] >> (8 * (e % 4)) & 15u) << (4 * w4_slot(e));
                    if (have) *reinterpret_cast<uint32_t *>(to) = n;
                }
                continue;
            }
            int b = sh.dim(c);                       // first byte of the lane's 8
            if constexpr (!I8) {
                // dims d and d + 16 share a byte: the lane of d takes the other's codes, two lanes on
#pragma unroll
                for (int h = 0; h < 2; ++h) w[c][h] |= (uint32_t)__shfl_xor((int)w[c][h], 2) << 4;
                b = b / 32 * 16 + b % 16;
            }
            turn(w[c][0], w[c][1]);
            if (quad < 16 && (I8 || (sh.l & 2) == 0)) {
                image[value_word(quad, b + 2 * sh.t4)] = w[c][0];
                image[value_word(quad, b + 2 * sh.t4 + 1)] = w[c][1];
            }
        }
    }
    if (!o.values) return;
    __syncthreads();
    uint8_t *to = part + codes + kv_code_bytes(FMT, in_page, D);
    for (int i = threadIdx.x; i < IMAGE / 16; i += kThreads) {
        const u4 s = *reinterpret_cast<const u4 *>(image + i * 4);
        const int m = i / 64 & 3;                    // how its dwords are turned: the same for a wave
        u4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = m == 0 ? s[q] : m == 1 ? s[q ^ 1] : m == 2 ? s[q ^ 2] : s[q ^ 3];
        if (o.lo == 0 && o.hi == 64) {
            *reinterpret_cast<u4 *>(to + i * 16) = w;
            continue;
        }
        // dword q holds the tokens 16 q + 4 (i / 16 % 4) .. + 3
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int t = 16 * q + i / 16 % 4 * 4;
            if (t >= o.lo && t + 4 <= o.hi) {
                *reinterpret_cast<uint32_t *>(to + i * 16 + q * 4) = w[q];
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (t + e >= o.lo && t + e < o.hi) to[i * 16 + q * 4 + e] = (uint8_t)(w[q] >> (8 * e));
        }
    }
}

template <int FMT, int D, bool BF16, bool PASSING>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvArgs a, uint16_t *k, int64_t k_stride, uint16_t *v,
                                                           int64_t v_stride, int blocks)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    typedef Share<D> S;
    constexpr int IMAGE = kv_code_bytes(FMT, 64, D), PIECES = (IMAGE / 16 + kThreads - 1) / kThreads;
    __shared__ __attribute__((aligned(16))) uint32_t image[IMAGE / 4];
    Block o;
    if (!kv_block(a, blocks, o)) return;
    const S sh(o);
    const int page_size = 1 << a.page_shift, in_page = (o.block * 64) & (page_size - 1);
    uint16_t *dst = o.values ? v : k;
    const int64_t stride = o.values ? v_stride : k_stride;
    const uint8_t *part = kv_part(a, max(o.page, 0), o.head);
    const int codes = kv_code_bytes(FMT, page_size, D);
    const float *arrays = reinterpret_cast<const float *>(part + 2 * codes) +
                          (o.values ? kv_arrays(FMT) / 2 * page_size : 0);
    float scale[S::ROUNDS], low[S::ROUNDS];
    uint32_t w[S::ROUNDS][S::CH][2];
    if (o.page >= 0) {
#pragma unroll
        for (int i = 0; i < S::ROUNDS; ++i) {
            const int t = sh.quad(i) * 4 + sh.t4;
            if (t < o.lo || t >= o.hi) continue;
            scale[i] = arrays[in_page + t];
            if constexpr (!I8) low[i] = arrays[page_size + in_page + t];
            if (!o.values)
#pragma unroll
                for (int c = 0; c < S::CH; ++c) {
                    const uint32_t *from = reinterpret_cast<const uint32_t *>(part + key_byte<FMT, D>(in_page + t, sh.dim(c)));
                    w[i][c][0] = from[0];
                    if constexpr (I8) w[i][c][1] = from[1];
                }
        }
        if (o.values) {
            const u4 *from = reinterpret_cast<const u4 *>(part + codes + kv_code_bytes(FMT, in_page, D));
            u4 s[PIECES];
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                const int i = p * kThreads + threadIdx.x;
                if (i < IMAGE / 16) s[p] = from[i];
            }
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                const int i = p * kThreads + threadIdx.x, m = i / 64 & 3;
                u4 u;
#pragma unroll
                for (int q = 0; q < 4; ++q) u[q] = m == 0 ? s[p][q] : m == 1 ? s[p][q ^ 1] : m == 2 ? s[p][q ^ 2] : s[p][q ^ 3];
                if (i < IMAGE / 16) *reinterpret_cast<u4 *>(image + i * 4) = u;
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < S::ROUNDS; ++i) {
        const int quad = sh.quad(i), t = quad * 4 + sh.t4;
        const bool have = t >= o.lo && t < o.hi;
        if (!__any(have)) break;
#pragma unroll
        for (int c = 0; c < S::CH; ++c) {
            us8 out = {0, 0, 0, 0, 0, 0, 0, 0};
            if (o.page >= 0) {
                if (o.values) {
                    const int b = I8 ? sh.dim(c) : sh.dim(c) / 32 * 16 + sh.dim(c) % 16, q = min(quad, 15);
                    w[i][c][0] = image[value_word(q, b + 2 * sh.t4)];
                    w[i][c][1] = image[value_word(q, b + 2 * sh.t4 + 1)];
                    turn_back(w[i][c][0], w[i][c][1]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float value;
                    if constexpr (I8) {
                        value = (float)((int)(w[i][c][e / 4] >> (8 * (e % 4)) & 255u) - 128) * scale[i];
                    } else {
                        const uint32_t n = o.values ? w[i][c][e / 4] >> (8 * (e % 4) + (sh.l & 2 ? 4 : 0))
                                                    : w[i][c][0] >> (4 * w4_slot(e));
                        value = __builtin_fmaf((float)(n & 15u), scale[i], low[i]);
                    }
                    out[e] = from_f32<BF16>(value);
                }
            }
            if (!have) continue;
            us8 *at = reinterpret_cast<us8 *>(dst + (o.row + t) * stride + o.head * D + sh.dim(c));
            if constexpr (PASSING) __builtin_nontemporal_store(out, at);
            else *at = out;
        }
    }
}

// Rows of more bytes than the L2 caches hold go past them (nontemporal): a prompt of 16384 rows, 8 heads of 128 dims, 8 bits,
// written and read back, 45.6 us for 50.6; 16 sequences of it read, 59 us for 66.  Few rows are in these caches, or wanted
// there, by the products before and after: 10.1 us so for 9.5 (32 rows).
constexpr int64_t kPassingBytes = 32 << 20;

// A launch of KERNEL<FMT, D, BF16, PASSING> for the sizes at hand
#define KV_LAUNCH(KERNEL, ...)                                                                      \
    do {                                                                                            \
        const int blocks = kv_blocks(a.max_rows);                                                   \
        const unsigned grid = (unsigned)((int64_t)a.count * blocks * 2 * a.heads);                  \
        auto go = [&](auto kernel) {                                                                \
            kernel<<<grid, kThreads, 0, s>>>(__VA_ARGS__, blocks);                                  \
            return hipGetLastError();                                                               \
        };                                                                                          \
        auto dims = [&](auto fmt, auto bf, auto far) {                                              \
            constexpr int F = decltype(fmt)::value;                                                 \
            constexpr bool B = decltype(bf)::value, P = decltype(far)::value;                       \
            return a.dim == 64 ? go(KERNEL<F, 64, B, P>)                                            \
                               : a.dim == 128 ? go(KERNEL<F, 128, B, P>) : go(KERNEL<F, 256, B, P>);\
        };                                                                                          \
        auto types = [&](auto fmt, auto far) {                                                      \
            return bf16 ? dims(fmt, std::true_type{}, far) : dims(fmt, std::false_type{}, far);     \
        };                                                                                          \
        auto formats = [&](auto far) {                                                              \
            return a.fmt == LOWBIT_KV_I8 ? types(std::integral_constant<int, LOWBIT_KV_I8>{}, far)  \
                                         : types(std::integral_constant<int, LOWBIT_KV_U4>{}, far); \
        };                                                                                          \
        const bool passing = (int64_t)a.rows * a.heads * a.dim * 4 > kPassingBytes;                 \
        return passing ? formats(std::true_type{}) : formats(std::false_type{});                    \
    } while (0)

}  // namespace

hipError_t launch_kv_write(const KvArgs &a, const void *kp, int64_t k_stride, const void *vp, int64_t v_stride,
                           int bf16, hipStream_t s)
{
    const uint16_t *k = static_cast<const uint16_t *>(kp), *v = static_cast<const uint16_t *>(vp);
    KV_LAUNCH(kv_write_kernel, a, k, k_stride, v, v_stride);
}

hipError_t launch_kv_read(const KvArgs &a, void *kp, int64_t k_stride, void *vp, int64_t v_stride, int bf16,
                          hipStream_t s)
{
    uint16_t *k = static_cast<uint16_t *>(kp), *v = static_cast<uint16_t *>(vp);
    KV_LAUNCH(kv_read_kernel, a, k, k_stride, v, v_stride);
}

}  // namespace lowbit
