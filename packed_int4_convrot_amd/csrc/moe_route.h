// Top-k selection of one row of router logits by one wave.
//
// Lane l holds the kNe consecutive logits from kNe l on as unsigned keys in
// the order of the floats (NaN and -inf are key 0: never chosen), so that in each
// of the k rounds the wave's maximum key, and among the lanes that hold it the
// lowest, give the largest logit at its lowest index.  The rounds depend on one
// another; a round is six shift-and-maximum steps, a ballot and the winner's scan
// of its own keys.  (Up to 64 experts, counting for each key the keys before it
// finds all slots at once, but measured no faster: 2.9 against 2.4 us for 5 tokens
// of 60, k = 4, and the same 4.5 us in front of the experts at k = 8.)
#pragma once

#include <type_traits>

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

// One row's logits and the slots chosen so far: lane j has slot j's expert (-1:
// none left) and its key.
template <int kNe>
struct Routed {
    uint32_t all[kNe];  // the keys of this lane's experts
    uint32_t top;
    uint32_t mine;
    int id;
};

// The first `rounds` slots of a row.
template <int kNe, bool kBf16>
__device__ __forceinline__ Routed<kNe> route_select(const void *row, int E, int rounds, int lane)
{
    Routed<kNe> r;
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kNe; ++i) {
        const int e = lane * kNe + i;
        r.all[i] = 0;
        if (e < E) {
            if constexpr (kBf16)
                r.all[i] = logit_key(bf16_to_f32(static_cast<const uint16_t *>(row)[e]));
            else
                r.all[i] = logit_key(static_cast<const float *>(row)[e]);
        }
    }
#pragma unroll
    for (int i = 0; i < kNe; ++i)
        if (r.all[i] > best)
            best = r.all[i], at = i;
    r.id = -1;
    r.mine = 0;
    r.top = wave_max(best);
    uint32_t m = r.top;
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        if (j > 0)
            m = wave_max(best);
        if (m == 0)
            break;
        const int src = __builtin_ctzll(__ballot(best == m));
        const int e = __builtin_amdgcn_readlane(lane * kNe + at, src);
        if (lane == j)
            r.id = e, r.mine = m;
        if (lane == src) {
            // Its next: the largest key after (m, gone) in the order of choice.
            best = 0;
            const int gone = at;
#pragma unroll
            for (int i = 0; i < kNe; ++i) {
                const bool left = r.all[i] < m || (r.all[i] == m && i > gone);
                if (left && r.all[i] > best)
                    best = r.all[i], at = i;
            }
        }
    }
    return r;
}

// Lane j's weight, of a row whose slots have all been chosen.
template <int kNe>
__device__ __forceinline__ float route_weight(const Routed<kNe> &r, bool renormalize)
{
    const float e = logit_exp(r.mine, r.top);
    float den = e;
    if (!renormalize) {
        den = 0.f;
#pragma unroll
        for (int i = 0; i < kNe; ++i) {
            den += logit_exp(r.all[i], r.top);
            if constexpr (kNe > 4)
                __builtin_amdgcn_sched_barrier(0);  // one exponential's registers at a time
        }
    }
    den = wave_sum(den);
    return den > 0.f ? e / den : 0.f;
}

// Calls f with the logits a lane holds for E experts.  One rule for the router and for
// the layer that routes its own tokens: the weights' sums run in an order that depends
// on it, and a token's weights should not depend on which of the two chose them.  (The
// fewest that fit: one token of a layer of H 2048, I 768, k 8 takes 15.4, 15.4 and 15.7 us
// with 32, 64 and 128 experts, against 17.1, 16.9 and 17.0 us with four logits a lane.)
template <class F>
auto with_lane_logits(int E, F &&f)
{
    if (E <= 64)
        return f(std::integral_constant<int, 1>());
    if (E <= 128)
        return f(std::integral_constant<int, 2>());
    if (E <= 256)
        return f(std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 16>());
}

}  // namespace ck
