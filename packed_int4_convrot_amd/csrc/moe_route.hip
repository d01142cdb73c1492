// Mixture-of-experts router: top-k of each token's logits, one wave a token.
// ids descending by logit, ties to the lowest expert; weights exp(l - max) over
// their sum (of the chosen, or of all experts), fp32.  Bound by launch latency
// for few tokens (5 tokens of 60 experts: 2.4 us) and for many by the rounds'
// instructions (8192 tokens, 8 of 256 fp32 logits: 11 us, of which eight waves a SIMD with
// 516 vector instructions each issue for 7; reading the 8 MB alone would take 2).
#include "moe_route.h"
#include "rows_launch.h"

namespace ck {
namespace {

constexpr int kTokensPerBlock = 4;

template <int kNe, bool kBf16>
__global__ __launch_bounds__(kTokensPerBlock * kWave) void moe_route_kernel(
    const void *__restrict__ logits, int64_t T, int E, int64_t ldl, int k, bool renormalize,
    int32_t *__restrict__ ids, float *__restrict__ weights)
{
    const int lane = threadIdx.x % kWave;
    const int64_t t = (int64_t)blockIdx.x * kTokensPerBlock + threadIdx.x / kWave;
    if (t >= T)
        return;
    const void *row = static_cast<const uint8_t *>(logits) + t * ldl * (kBf16 ? 2 : 4);
    const Routed<kNe> r = route_select<kNe, kBf16>(row, E, k, lane);
    const float w = route_weight(r, renormalize);
    if (lane < k) {
        ids[t * k + lane] = r.id;
        weights[t * k + lane] = w;
    }
}

template <bool kBf16>
void launch_kind(const void *logits, int64_t T, int E, int64_t ldl, int k, bool renormalize, int32_t *ids,
                 float *weights, hipStream_t s)
{
    const dim3 grid((unsigned)((T + kTokensPerBlock - 1) / kTokensPerBlock)), block(kTokensPerBlock * kWave);
    with_lane_logits(E, [&](auto ne) {
        hipLaunchKernelGGL((moe_route_kernel<decltype(ne)::value, kBf16>), grid, block, 0, s, logits, T, E, ldl, k,
                           renormalize, ids, weights);
    });
}

}  // namespace

int launch_moe_route(const void *logits, bool bf16, int64_t T, int E, int64_t ldl, int k, bool renormalize,
                     int32_t *ids, float *weights, void *stream)
{
    if (T <= 0)
        return 0;
    if (E < 1 || E > kRouteMaxExperts || k < 1 || k > kRouteMaxK)
        return (int)hipErrorInvalidValue;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (bf16)
        launch_kind<true>(logits, T, E, ldl, k, renormalize, ids, weights, s);
    else
        launch_kind<false>(logits, T, E, ldl, k, renormalize, ids, weights, s);
    return (int)hipGetLastError();
}

}  // namespace ck
