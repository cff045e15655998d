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
#include "lowbit_internal.hpp"

namespace lowbit {

namespace {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void put(void *y, int64_t o, float v, int bf16)
{
    if (bf16)
        static_cast<__bf16 *>(y)[o] = (__bf16)v;
    else
        static_cast<_Float16 *>(y)[o] = (_Float16)v;
}

// 16 bytes of a row at K offset k; bytes past K (a multiple of 8) are zeros
__device__ __forceinline__ i4 row16(const int8_t *row, int k, int K)
{
    i2 lo = {0, 0}, hi = {0, 0};
    if (k < K) lo = *reinterpret_cast<const i2 *>(row + k);
    if (k + 8 < K) hi = *reinterpret_cast<const i2 *>(row + k + 8);
    return i4{lo.x, lo.y, hi.x, hi.y};
}

// ---------------------------------------------------------------- streaming
// One workgroup per 16 channels; its 8 waves split K into runs of 64-byte
// chunks and add their int32 partial sums through LDS.  Rows past the last
// (of the activation or the weight) are read as copies of the last one and
// not stored.
constexpr int kStreamWaves = 8;

template <bool GROUPED>
__global__ __launch_bounds__(kStreamWaves * 64)
void w8a8_stream_kernel(W8Args p)
{
    __shared__ int part[kStreamWaves][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r16 = lane & 15, kq = lane >> 4;
    const int n0 = blockIdx.x * 16;
    int first = 0, last = p.rows;
    const int8_t *w = p.w;
    const float *ws = p.ws;
    if constexpr (GROUPED) {
        const int e = blockIdx.y;
        first = max(p.offsets[e], 0);
        last = min(p.offsets[e + 1], p.rows);
        w += (int64_t)e * p.N * p.K;
        ws += (int64_t)e * p.N;
    }
    const int8_t *wr = w + (int64_t)min(n0 + r16, p.N - 1) * p.K;
    const int full = p.K / 64;                        // whole 64-byte chunks
    const int per = (full + kStreamWaves - 1) / kStreamWaves;
    const int c0 = min(wave * per, full), c1 = min(c0 + per, full);
    const int step = GROUPED ? 16 : 16 * gridDim.y;
    for (int m0 = first + (GROUPED ? 0 : 16 * (int)blockIdx.y); m0 < last; m0 += step) {
        const int64_t src = w8a8_source_row(p, min(m0 + r16, last - 1));
        const int8_t *xr = p.x + src * p.K;
        i4 acc = {0, 0, 0, 0};
#pragma unroll 4
        for (int c = c0; c < c1; ++c) {
            const int k = c * 64 + kq * 16;
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(row16(wr, k, p.K), row16(xr, k, p.K), acc, 0, 0, 0);
        }
        if (wave == kStreamWaves - 1 && full * 64 < p.K) {
            const int k = full * 64 + kq * 16;
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(row16(wr, k, p.K), row16(xr, k, p.K), acc, 0, 0, 0);
        }
        // lane: token r16, channels 4 kq .. 4 kq + 3
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][r16 * 16 + kq * 4 + i] = acc[i];
        __syncthreads();
        if (tid < 256) {
            int s = 0;
#pragma unroll
            for (int q = 0; q < kStreamWaves; ++q) s += part[q][tid];
            const int m = m0 + (tid >> 4), n = n0 + (tid & 15);
            if (m < last && n < p.N) {
                float v = (float)s * p.xs[w8a8_source_row(p, m)] * ws[n];
                if (p.bias) v += p.bias[n];
                put(p.y, (int64_t)m * p.N + n, v, p.y_bf16);
            }
        }
        __syncthreads();
    }
}

}  // namespace

size_t gemm_w8a8_workspace(int, int, int) { return 0; }

hipError_t launch_gemm_w8a8(const W8Args &a, void *, hipStream_t s)
{
    const dim3 grid((a.N + 15) / 16, a.rows / 16 + 1 < 65535 ? (a.rows + 15) / 16 : 65535);
    w8a8_stream_kernel<false><<<grid, kStreamWaves * 64, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_gemm_w8a8(const W8Args &a, hipStream_t s)
{
    w8a8_stream_kernel<true><<<dim3((a.N + 15) / 16, a.E), kStreamWaves * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace lowbit
