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
// for the keys or the values of one head; dim / 8 lanes hold a row, 8 values
// each.  A row of keys goes to memory in pieces of 8 (4) bytes as it is.  The
// page holds values by dim, 4 tokens to a dword, so they are turned in LDS, in
// the page's own byte order, and leave it 16 bytes at a time where the block is
// whole, by dwords and bytes at its ends: no byte of another token is written.
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

// Byte of (token t, first dim d of 8) in a page's keys, and of (token t, dim d)
// in a block of values (4 bits: d counts bytes: 16 of every 32 dims)
template <int FMT, int D>
__device__ __forceinline__ int key_byte(int t, int d)
{
    if (FMT == LOWBIT_KV_I8) return ((t / 16 * (D / 64) + d / 64) * 4 + d % 64 / 16) * 256 + t % 16 * 16 + d % 16;
    return ((t / 32 * (D / 64) + d / 64) * 4 + d % 64 / 16) * 256 + t % 16 * 16 + t % 32 / 16 * 8 + d % 16 / 8 * 4;
}
__device__ __forceinline__ int value_byte(int t, int d)
{
    return (d / 16 * 4 + t % 16 / 4) * 256 + d % 16 * 16 + t / 16 * 4 + t % 4;
}

template <int LANES, typename T, typename F>
__device__ __forceinline__ T across(T v, F f)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = f(v, (T)__shfl_xor(v, o));
    return v;
}

template <int FMT, int D, bool BF16>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvArgs a, const uint16_t *k, int64_t k_stride,
                                                            const uint16_t *v, int64_t v_stride, int blocks)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    constexpr int LANES = D / 8, STEP = kThreads / LANES, IMAGE = kv_code_bytes(FMT, 64, D);
    __shared__ __attribute__((aligned(16))) uint8_t image[IMAGE];
    Block o;
    if (!kv_block(a, blocks, o) || o.page < 0) return;
    const int tid = threadIdx.x, l = tid % LANES;
    const int page_size = 1 << a.page_shift, in_page = (o.block * 64) & (page_size - 1);
    uint8_t *part = kv_part(a, o.page, o.head);
    const int codes = kv_code_bytes(FMT, page_size, D);
    float *arrays = reinterpret_cast<float *>(part + 2 * codes) + (o.values ? kv_arrays(FMT) / 2 * page_size : 0);
    const uint16_t *src = o.values ? v : k;
    const int64_t stride = o.values ? v_stride : k_stride;

    for (int t0 = o.lo; t0 < o.hi; t0 += STEP) {
        const int t = t0 + tid / LANES;
        const bool have = t < o.hi;
        us8 raw = {0, 0, 0, 0, 0, 0, 0, 0};
        if (have) raw = *reinterpret_cast<const us8 *>(src + (o.row + t) * stride + o.head * D + l * 8);
        float x[8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = to_f32<BF16>(raw[i]);
            top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
        }
        top = across<LANES>(top, [](uint32_t p, uint32_t q) { return max(p, q); });
        const bool bad = top >= 0x7f800000u;         // an infinity or a NaN
        float scale, low = 0.f;
        uint32_t code[8];
        if constexpr (I8) {
            const float amax = __uint_as_float(top), inv = fminf(127.f / amax, FLT_MAX);
            scale = amax / 127.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) code[i] = bad ? 128u : (uint32_t)((int)rintf(x[i] * inv) + 128);
        } else {
            float lo = x[0], hi = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                lo = fminf(lo, x[i]);
                hi = fmaxf(hi, x[i]);
            }
            lo = across<LANES>(lo, [](float p, float q) { return fminf(p, q); });
            hi = across<LANES>(hi, [](float p, float q) { return fmaxf(p, q); });
            const float h = 0.5f * hi - 0.5f * lo, inv = fminf(15.f / h, FLT_MAX);
            scale = h / 7.5f;
            low = bad ? 0.f : lo;
#pragma unroll
            for (int i = 0; i < 8; ++i) code[i] = bad ? 0u : (uint32_t)(int)rintf((0.5f * x[i] - 0.5f * lo) * inv);
        }
        if (have && l == 0) {
            const int at = in_page + t;
            arrays[at] = bad ? __uint_as_float(0x7fc00000u) : scale;
            if constexpr (!I8) arrays[page_size + at] = low;
        }
        if (!o.values) {
            uint8_t *to = part + key_byte<FMT, D>(in_page + t, l * 8);
            if constexpr (I8) {
                const uint2 w = {code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24,
                                 code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24};
                if (have) *reinterpret_cast<uint2 *>(to) = w;
            } else {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) w |= code[i] << (4 * w4_slot(i));
                if (have) *reinterpret_cast<uint32_t *>(to) = w;
            }
        } else if constexpr (I8) {
            if (have)
#pragma unroll
                for (int i = 0; i < 8; ++i) image[value_byte(t, l * 8 + i)] = (uint8_t)code[i];
        } else {
            // dim d and dim d + 16 share a byte: the lane of d takes the other's codes from two lanes on
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = code[i] | (uint32_t)__shfl_xor((int)code[i], 2) << 4;
                if (have && (l & 2) == 0) image[value_byte(t, l / 4 * 16 + (l & 1) * 8 + i)] = (uint8_t)w;
            }
        }
    }
    if (!o.values) return;
    __syncthreads();
    uint8_t *to = part + codes + kv_code_bytes(FMT, in_page, D);
    for (int i = tid; i < IMAGE / 16; i += kThreads) {
        const u4 w = *reinterpret_cast<const u4 *>(image + i * 16);
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

template <int FMT, int D, bool BF16>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvArgs a, uint16_t *k, int64_t k_stride, uint16_t *v,
                                                           int64_t v_stride, int blocks)
{
    constexpr bool I8 = FMT == LOWBIT_KV_I8;
    constexpr int LANES = D / 8, STEP = kThreads / LANES, IMAGE = kv_code_bytes(FMT, 64, D);
    __shared__ __attribute__((aligned(16))) uint8_t image[IMAGE];
    Block o;
    if (!kv_block(a, blocks, o)) return;
    const int tid = threadIdx.x, l = tid % LANES;
    const int page_size = 1 << a.page_shift, in_page = (o.block * 64) & (page_size - 1);
    uint16_t *dst = o.values ? v : k;
    const int64_t stride = o.values ? v_stride : k_stride;
    if (o.page < 0) {
        const us8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int t = o.lo + tid / LANES; t < o.hi; t += STEP)
            *reinterpret_cast<us8 *>(dst + (o.row + t) * stride + o.head * D + l * 8) = zero;
        return;
    }
    const uint8_t *part = kv_part(a, o.page, o.head);
    const int codes = kv_code_bytes(FMT, page_size, D);
    const float *arrays = reinterpret_cast<const float *>(part + 2 * codes) +
                          (o.values ? kv_arrays(FMT) / 2 * page_size : 0);
    if (o.values) {
        const uint8_t *from = part + codes + kv_code_bytes(FMT, in_page, D);
        for (int i = tid; i < IMAGE / 16; i += kThreads)
            *reinterpret_cast<u4 *>(image + i * 16) = *reinterpret_cast<const u4 *>(from + i * 16);
        __syncthreads();
    }
    for (int t = o.lo + tid / LANES; t < o.hi; t += STEP) {
        const float scale = arrays[in_page + t], low = I8 ? 0.f : arrays[page_size + in_page + t];
        us8 out;
        uint32_t w[2] = {0, 0};
        if (!o.values) {
            const uint8_t *from = part + key_byte<FMT, D>(in_page + t, l * 8);
            w[0] = *reinterpret_cast<const uint32_t *>(from);
            if constexpr (I8) w[1] = *reinterpret_cast<const uint32_t *>(from + 4);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t c;
            if constexpr (I8)
                c = o.values ? image[value_byte(t, l * 8 + i)] : (w[i / 4] >> (8 * (i % 4))) & 255;
            else
                c = (o.values ? image[value_byte(t, l / 4 * 16 + (l & 1) * 8 + i)] >> (l & 2 ? 4 : 0)
                              : w[0] >> (4 * w4_slot(i))) & 15;
            const float value = I8 ? (float)((int)c - 128) * scale : __builtin_fmaf((float)c, scale, low);
            out[i] = from_f32<BF16>(value);
        }
        *reinterpret_cast<us8 *>(dst + (o.row + t) * stride + o.head * D + l * 8) = out;
    }
}

// A launch of KERNEL<FMT, D, BF16> for the sizes at hand
#define KV_LAUNCH(KERNEL, ...)                                                                      \
    do {                                                                                            \
        const int blocks = kv_blocks(a.max_rows);                                                   \
        const unsigned grid = (unsigned)((int64_t)a.count * blocks * 2 * a.heads);                  \
        auto go = [&](auto kernel) {                                                                \
            kernel<<<grid, kThreads, 0, s>>>(__VA_ARGS__, blocks);                                  \
            return hipGetLastError();                                                               \
        };                                                                                          \
        auto dims = [&](auto fmt, auto bf) {                                                        \
            constexpr int F = decltype(fmt)::value;                                                 \
            constexpr bool B = decltype(bf)::value;                                                 \
            return a.dim == 64 ? go(KERNEL<F, 64, B>)                                               \
                               : a.dim == 128 ? go(KERNEL<F, 128, B>) : go(KERNEL<F, 256, B>);      \
        };                                                                                          \
        using i8 = std::integral_constant<int, LOWBIT_KV_I8>;                                       \
        using u4b = std::integral_constant<int, LOWBIT_KV_U4>;                                      \
        if (a.fmt == LOWBIT_KV_I8) return bf16 ? dims(i8{}, std::true_type{}) : dims(i8{}, std::false_type{});  \
        return bf16 ? dims(u4b{}, std::true_type{}) : dims(u4b{}, std::false_type{});               \
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
