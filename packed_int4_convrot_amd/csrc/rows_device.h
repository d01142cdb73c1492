// Device helpers of the mixture-of-experts and adapter kernels.
#pragma once

#include "ck_device.h"

namespace ck {

// Eight packed codes (one dword, nibble i = column i) as bf16 128 + q: the bit
// pattern 0x4300 | q.  Pairs come out in the column order (0,4) (1,5) (2,6)
// (3,7), two operations a pair; act_order8() puts activations in the same order.
__device__ __forceinline__ v8bf w4_bf16_plus128(uint32_t d)
{
    // The mask in a vector and the pattern in a scalar register, for v_and_or_b32
    // (an instruction takes one scalar operand).
    uint32_t mask = 0x000f000fu, pattern = 0x43004300u;
    asm("" : "+v"(mask));
    asm("" : "+s"(pattern));
    u32x4 r;
    r[0] = (d & mask) | pattern;
    r[1] = ((d >> 4) & mask) | pattern;
    r[2] = ((d >> 8) & mask) | pattern;
    r[3] = ((d >> 12) & mask) | pattern;
    return __builtin_bit_cast(v8bf, r);
}

// Eight consecutive bf16 in the column order of w4_bf16_plus128().
__device__ __forceinline__ v8bf act_order8(u32x4 w)
{
    u32x4 r;
    r[0] = perm(w[2], w[0], 0x05040100u);
    r[1] = perm(w[2], w[0], 0x07060302u);
    r[2] = perm(w[3], w[1], 0x05040100u);
    r[3] = perm(w[3], w[1], 0x07060302u);
    return __builtin_bit_cast(v8bf, r);
}
// 16 x 16 x 32 bf16 MFMA.  Lane l holds row (a) or column (b) l % 16 and the 8
// k-values of quarter l / 16; the result's lane l holds column l % 16, rows
// 4 (l / 16) + i.
__device__ __forceinline__ v4f mfma16(v8bf a, v8bf b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// fp32 as the sum of two bf16: 16 significant bits.  The second part of a
// value whose first is not finite is 0, so that infinities stay infinities.
__device__ __forceinline__ void split_bf16(float v, uint16_t &hi, uint16_t &lo)
{
    hi = f32_to_bf16(v);
    const float h = bf16_to_f32(hi);
    lo = (hi & 0x7f80u) == 0x7f80u ? (uint16_t)0 : f32_to_bf16(v - h);
}

// Maximum over the wave by data-parallel-primitive shifts; lane 63 has it.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, dpp_or_zero<0x111, 0xf>(v));  // row_shr:1
    v = max(v, dpp_or_zero<0x112, 0xf>(v));
    v = max(v, dpp_or_zero<0x114, 0xf>(v));
    v = max(v, dpp_or_zero<0x118, 0xf>(v));
    v = max(v, dpp_or_zero<0x142, 0xa>(v));  // row_bcast:15
    v = max(v, dpp_or_zero<0x143, 0xc>(v));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// Sums over the lanes up to each, the same way; lane 63 has the wave's.
template <int kCtrl, int kRows>
__device__ __forceinline__ int dpp_add(int v)
{
    return v + (int)dpp_or_zero<kCtrl, kRows>((uint32_t)v);
}
__device__ __forceinline__ int wave_scan(int v)
{
    v = dpp_add<0x111, 0xf>(v);
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);
    return dpp_add<0x143, 0xc>(v);
}
// Sum over the wave, in a fixed order.
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

}  // namespace ck
