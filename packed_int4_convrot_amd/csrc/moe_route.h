// Top-k selection of one row of router logits by one wave.
//
// Lane l holds the kNe consecutive logits from kNe l on as unsigned keys in
// the order of the floats (NaN and -inf are key 0: never chosen), so that in each
// of the k rounds the wave's maximum key, and among the lanes that hold it the
// lowest, give the largest logit at its lowest index.  The rounds depend on one
// another; a round is six fused shift-and-maximum operations and a ballot.
#pragma once

#include "rows_device.h"

namespace ck {

__device__ __forceinline__ uint32_t logit_key(float v)
{
    v += 0.f;  // -0 ties with +0
    const uint32_t u = __float_as_uint(v);
    if (!(v > -INFINITY))  // -inf or NaN
        return 0;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
// exp(l - top); where top is +inf, the +inf logits share the weight.
__device__ __forceinline__ float logit_exp(uint32_t key, uint32_t top)
{
    const float m = key_logit(top), l = key_logit(key);
    if (key == 0)
        return 0.f;
    return m == INFINITY ? (l == INFINITY ? 1.f : 0.f) : expf(l - m);
}

// On return lane j < k has slot j's expert (-1: none left) and weight.
template <int kNe, bool kBf16>
__device__ __forceinline__ void route_row(const void *row, int E, int k, bool renormalize, int lane, int &id,
                                          float &weight)
{
    uint32_t key[kNe];
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kNe; ++i) {
        const int e = lane * kNe + i;
        key[i] = 0;
        if (e < E) {
            if constexpr (kBf16)
                key[i] = logit_key(bf16_to_f32(static_cast<const uint16_t *>(row)[e]));
            else
                key[i] = logit_key(static_cast<const float *>(row)[e]);
        }
    }
#pragma unroll
    for (int i = 0; i < kNe; ++i)
        if (key[i] > best)
            best = key[i], at = i;
    const uint32_t top = wave_max(best);
    float all = 0.f;
    if (!renormalize) {
#pragma unroll
        for (int i = 0; i < kNe; ++i) {
            all += logit_exp(key[i], top);
            if constexpr (kNe > 4)
                __builtin_amdgcn_sched_barrier(0);  // one exponential's registers at a time
        }
        all = wave_sum(all);
    }
    id = -1;
    uint32_t mine = 0;
    uint32_t m = top;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        if (j > 0)
            m = wave_max(best);
        if (m == 0)
            break;
        const int src = __builtin_ctzll(__ballot(best == m));
        const int e = __builtin_amdgcn_readlane(lane * kNe + at, src);
        if (lane == j)
            id = e, mine = m;
        if (lane == src) {
            // Its next: the largest key after (m, gone) in the order of choice.
            best = 0;
            const int gone = at;
#pragma unroll
            for (int i = 0; i < kNe; ++i) {
                const bool left = key[i] < m || (key[i] == m && i > gone);
                if (left && key[i] > best)
                    best = key[i], at = i;
            }
        }
    }
    const float e = logit_exp(mine, top);
    const float den = renormalize ? wave_sum(e) : all;
    weight = den > 0.f ? e / den : 0.f;
}

}  // namespace ck
