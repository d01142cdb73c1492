// Quantisers to e4m3 with power-of-two scales (e8m0) for each block of 128: activations
// (a scale for each row and 128 columns), weights (128 x 128), and the weights' transposer.
//
// A block's scale is the smallest power of two that keeps its values within 448, so x / s
// is exact and the code is x's own nearest e4m3 value: one rounding.
//
// All are bound by memory: one pass, 16 columns a lane, whole lines either way.  8192 rows of 10240
// columns take 44 us (252 MB, 5.7 TB/s), 2000 of 2048 5.3, five of 3840 2.6 (a launch); a weight of
// 20480 x 3840 40 us (236 MB, 5.8 TB/s), its transpose 29 to 35 (157 MB, 4.5 to 5.3 TB/s; LDS bytes
// are gathered across rows, whose conflicts hide under the loads).
#include "fp8_device.h"
#include "fp8_launch.h"

namespace ck {
namespace {

constexpr int kThreads = 256;
constexpr int kLaneColumns = 16;
constexpr int kRowsEach = kThreads / kWave;     // of a workgroup
constexpr int kSegment = kWave * kLaneColumns;  // columns of a wave: eight blocks

__device__ __forceinline__ float abs_max16(const float (&v)[16])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        a = fmaxf(a, fabsf(v[i]));
    return a;
}

// The same by the values' bits, in which a NaN is above all others (fmaxf leaves it out).
__device__ __forceinline__ uint32_t abs_max16_bits(const float (&v)[16])
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
    return a;
}

__device__ __forceinline__ u32x4 codes16(const float (&v)[16], float scale)
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = pack_e4m3x4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], scale);
    return r;
}

template <bool kF32>
__device__ __forceinline__ void load16(const void *x, int64_t at, float (&v)[16])
{
    if constexpr (kF32) {
        const v4f *p = reinterpret_cast<const v4f *>(static_cast<const float *>(x) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const v4f w = p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[4 * i + j] = w[j];
        }
    } else {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 w = p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = bf16_to_f32(w[j] & 0xffffu);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
}

// A wave quantises 1024 columns of a row, a lane 16 of them; eight lanes share a block.  (x, the
// segments of a row, by y, rows: a division would take a third of the time of a few rows.)
template <bool kF32>
__global__ __launch_bounds__(kThreads) void fp8_quant_kernel(const void *__restrict__ x, int64_t M, int K, int64_t ldx,
                                                             uint8_t *__restrict__ codes, int64_t lda,
                                                             uint8_t *__restrict__ scales, int64_t ldsa)
{
    const int lane = threadIdx.x % kWave;
    const int k = blockIdx.x * kSegment + lane * kLaneColumns;
    for (int64_t m = blockIdx.y * kRowsEach + threadIdx.x / kWave; m < M; m += (int64_t)gridDim.y * kRowsEach) {
        float v[16];
        if (k < K) {
            load16<kF32>(x, m * ldx + k, v);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = 0.f;
        }
        float a = abs_max16(v);
        a = fmaxf(a, __shfl_xor(a, 1));
        a = fmaxf(a, __shfl_xor(a, 2));
        a = fmaxf(a, __shfl_xor(a, 4));
        const uint32_t s = e8m0_of(a);
        if (k < K) {
            *reinterpret_cast<u32x4 *>(codes + m * lda + k) = codes16(v, e8m0_value(s));
            if (lane % 8 == 0)
                scales[m * ldsa + k / kFp8Block] = (uint8_t)s;
        }
    }
}

// One 128 x 128 block a workgroup: a thread holds 16 columns of four rows.  A NaN gives the block the
// scale NaN, as an infinity does: a row of activations is spoiled by its NaN code alone, but here the
// block's other outputs would stay finite.
__global__ __launch_bounds__(kThreads) void fp8_weight_kernel(const uint16_t *__restrict__ w, int N, int K,
                                                              int64_t ldw_in, uint8_t *__restrict__ codes, int64_t ldw,
                                                              uint8_t *__restrict__ scales)
{
    __shared__ uint32_t part[kThreads / kWave];
    const int bn = blockIdx.y, bk = blockIdx.x;
    const int k = bk * kFp8Block + threadIdx.x % 8 * kLaneColumns;
    float v[4][16];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = bn * kFp8Block + i * 32 + threadIdx.x / 8;
        if (n < N && k < K) {
            load16<false>(w, n * ldw_in + k, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[i][j] = 0.f;
        }
        a = max(a, abs_max16_bits(v[i]));
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        a = max(a, (uint32_t)__shfl_xor((int)a, d));
    if (threadIdx.x % kWave == 0)
        part[threadIdx.x / kWave] = a;
    __syncthreads();
    a = max(max(part[0], part[1]), max(part[2], part[3]));
    const uint32_t s = e8m0_of(__uint_as_float(a));
    const float by = e8m0_value(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = bn * kFp8Block + i * 32 + threadIdx.x / 8;
        if (n < N && k < K)
            *reinterpret_cast<u32x4 *>(codes + n * ldw + k) = codes16(v[i], by);
    }
    if (threadIdx.x == 0)
        scales[(int64_t)bn * gridDim.x + bk] = (uint8_t)s;
}

// One 128 x 128 block a workgroup through LDS, whose rows are padded by one dword.
__global__ __launch_bounds__(kThreads) void fp8_transpose_kernel(const uint8_t *__restrict__ codes, int64_t ldw,
                                                                 const uint8_t *__restrict__ scales, int N, int K,
                                                                 uint8_t *__restrict__ codes_t, int64_t ldt,
                                                                 uint8_t *__restrict__ scales_t)
{
    constexpr int kPitch = kFp8Block + 4;
    __shared__ uint32_t tile[kFp8Block * kPitch / 4];
    const int bn = blockIdx.y, bk = blockIdx.x, c = threadIdx.x % 8 * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 32 + threadIdx.x / 8, n = bn * kFp8Block + r, k = bk * kFp8Block + c;
        if (n < N && k < K) {
            const u32x4 q = *reinterpret_cast<const u32x4 *>(codes + n * ldw + k);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                tile[(r * kPitch + c) / 4 + j] = q[j];
        }
    }
    __syncthreads();
    const uint8_t *bytes = reinterpret_cast<const uint8_t *>(tile);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 32 + threadIdx.x / 8, k = bk * kFp8Block + r, n = bn * kFp8Block + c;
        if (n < N && k < K) {
            u32x4 q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[j] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    q[j] |= (uint32_t)bytes[(c + 4 * j + b) * kPitch + r] << 8 * b;
            }
            *reinterpret_cast<u32x4 *>(codes_t + k * ldt + n) = q;
        }
    }
    if (threadIdx.x == 0)
        scales_t[(int64_t)bk * gridDim.y + bn] = scales[(int64_t)bn * gridDim.x + bk];
}

}  // namespace

int launch_fp8_quant(const void *x, bool f32, int64_t M, int K, int64_t ldx, uint8_t *codes, int64_t lda,
                     uint8_t *scales, int64_t ldsa, void *stream)
{
    if (M <= 0)
        return 0;
    const int segments = (K + kSegment - 1) / kSegment;
    auto kern = f32 ? fp8_quant_kernel<true> : fp8_quant_kernel<false>;
    constexpr int64_t kMostRuns = 65535;
    const int64_t runs = (M + kRowsEach - 1) / kRowsEach;
    hipLaunchKernelGGL(kern, dim3((unsigned)segments, (unsigned)(runs < kMostRuns ? runs : kMostRuns)), dim3(kThreads),
                       0, reinterpret_cast<hipStream_t>(stream), x, M, K, ldx, codes, lda, scales, ldsa);
    return (int)hipGetLastError();
}

int launch_fp8_quantize_weights(const uint16_t *w, int64_t N, int K, int64_t ldw_in, uint8_t *codes, int64_t ldw,
                                uint8_t *scales, void *stream)
{
    if (N <= 0)
        return 0;
    hipLaunchKernelGGL(fp8_weight_kernel, dim3((unsigned)fp8_blocks(K), (unsigned)fp8_blocks(N)), dim3(kThreads), 0,
                       reinterpret_cast<hipStream_t>(stream), w, (int)N, K, ldw_in, codes, ldw, scales);
    return (int)hipGetLastError();
}

int launch_fp8_transpose(const uint8_t *codes, int64_t ldw, const uint8_t *scales, int N, int K, uint8_t *codes_t,
                         int64_t ldt, uint8_t *scales_t, void *stream)
{
    hipLaunchKernelGGL(fp8_transpose_kernel, dim3((unsigned)fp8_blocks(K), (unsigned)fp8_blocks(N)), dim3(kThreads), 0,
                       reinterpret_cast<hipStream_t>(stream), codes, ldw, scales, N, K, codes_t, ldt, scales_t);
    return (int)hipGetLastError();
}

}  // namespace ck
