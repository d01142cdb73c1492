// C ABI of the operators that choose weights row by row: the mixture-of-experts
// router and layer, and the low-rank adapters.  Validation and dispatch as in
// ck_api.cpp: nothing is enqueued until every check has passed.  Semantics are
// documented in include/ck.h.
#include "../../include/ck.h"

#include "api_check.h"
#include "rows_launch.h"

namespace {

using namespace ck::api;

int check_logits(const char *fn, const void *logits, int32_t kind, int64_t E, int64_t ldl)
{
    if (kind != CK_LOGITS_F32 && kind != CK_LOGITS_BF16)
        return fail(CK_ERR_INVALID_ARG, "%s: unknown logit kind %d", fn, kind);
    if (!logits || !aligned(logits, kind == CK_LOGITS_BF16 ? 2 : 4))
        return fail(CK_ERR_INVALID_ARG, "%s: logits must be a non-NULL aligned pointer", fn);
    if (ldl < E)
        return fail(CK_ERR_INVALID_ARG, "%s: ldl (%lld) must be >= E (%lld)", fn, (long long)ldl, (long long)E);
    return CK_OK;
}

int check_routing(const char *fn, int64_t E, int32_t k)
{
    if (E < 1 || k < 1)
        return fail(CK_ERR_INVALID_ARG, "%s: E and k must be positive (E=%lld, k=%d)", fn, (long long)E, k);
    if (E > ck::kRouteMaxExperts || k > ck::kRouteMaxK)
        return fail(CK_ERR_UNSUPPORTED, "%s: takes E <= %d and k <= %d (E=%lld, k=%d)", fn, ck::kRouteMaxExperts,
                    ck::kRouteMaxK, (long long)E, k);
    return CK_OK;
}

int check_slots(const char *fn, const int32_t *ids, const float *weights)
{
    if (!ids || !aligned(ids, 4) || !weights || !aligned(weights, 4))
        return fail(CK_ERR_INVALID_ARG, "%s: ids and weights must be non-NULL 4-byte aligned pointers", fn);
    return CK_OK;
}

int64_t logit_size(int32_t kind) { return kind == CK_LOGITS_BF16 ? 2 : 4; }

int ck_moe_route_impl(const void *logits, int32_t kind, int64_t T, int64_t E, int64_t ldl, int32_t k,
                      int32_t renormalize, int32_t *ids, float *weights, void *stream)
{
    const char *fn = "ck_moe_route";
    CK_TRY(check_m(fn, T));
    CK_TRY(check_routing(fn, E, k));
    if (T == 0)
        return ok();
    CK_TRY(check_logits(fn, logits, kind, E, ldl));
    CK_TRY(check_slots(fn, ids, weights));
    const Range rl = span(logits, T, E, ldl, logit_size(kind));
    const Range ri = span(ids, T, k, k, 4), rw = span(weights, T, k, k, 4);
    if (overlap(rl, ri) || overlap(rl, rw) || overlap(ri, rw))
        return fail(CK_ERR_INVALID_ARG, "%s: logits, ids and weights must not overlap", fn);
    return hip_status(ck::launch_moe_route(logits, kind == CK_LOGITS_BF16, T, (int)E, ldl, k, renormalize != 0, ids,
                                           weights, stream),
                      fn);
}

// The workspace of T tokens holds P pairs at H <= 8192; a wider layer takes fewer
// tokens a pass (one at least: k <= 32 pairs of H <= 32768 need four times k pairs' room).
int64_t moe_room_pairs(int64_t T, int32_t k)
{
    const int64_t most = ck::kMoePairs / k * k, P = T * k < most ? T * k : most;
    return P < 4 * k ? 4 * k : P;
}

size_t moe_workspace(int64_t T, int64_t I, int64_t E, int32_t k)
{
    if (T <= 0 || I <= 0 || I % 64 != 0 || E < 1 || E > ck::kRouteMaxExperts || k < 1 || k > ck::kRouteMaxK || I > kMaxK ||
        T > kMaxRows)
        return 0;
    const int64_t P = moe_room_pairs(T, k);
    return (size_t)ck::moe_hidden_bytes(P, I) + (size_t)ck::moe_pass_columns(P) * 4;
}

// Tokens of one pass: the pairs a pass takes, and the results its room holds.
int64_t moe_pass_tokens(int64_t T, int64_t H, int32_t k)
{
    const int64_t by_pairs = ck::kMoePairs / k;
    const int64_t by_room = ck::moe_pass_columns(moe_room_pairs(T, k)) / H / k;
    const int64_t n = by_pairs < by_room ? by_pairs : by_room;
    return T < n ? T : n;
}

// logits null: ids and weights are inputs.
int moe_common(const char *fn, const uint16_t *x, int64_t T, int64_t H, int64_t ldx, const void *logits,
               int32_t kind, int64_t ldl, int32_t renormalize, bool routed, int32_t *ids, float *weights, int32_t k,
               int64_t E, int64_t I, int32_t Gw, const uint8_t *w1, const uint16_t *s1, const uint16_t *z1,
               const uint8_t *w2, const uint16_t *s2, const uint16_t *z2, uint16_t *out, int64_t ldo, void *ws,
               size_t ws_bytes, void *stream)
{
    CK_TRY(check_m(fn, T));
    CK_TRY(check_k(fn, H));
    CK_TRY(check_routing(fn, E, k));
    if (I <= 0 || I % 64 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: I must be a positive multiple of 64 (got %lld)", fn, (long long)I);
    if (I > kMaxK)
        return fail(CK_ERR_UNSUPPORTED, "%s: I must be at most %lld (got %lld)", fn, (long long)kMaxK, (long long)I);
    if (Gw != 64)
        return fail(CK_ERR_UNSUPPORTED, "%s: needs Gw == 64 (got %d)", fn, Gw);
    if (!w1 || !s1 || !w2 || !s2)
        return fail(CK_ERR_INVALID_ARG, "%s: expert weights and scales must not be NULL", fn);
    if (!aligned(w1, 16) || !aligned(s1, 16) || !aligned(z1, 16) || !aligned(w2, 16) || !aligned(s2, 16) ||
        !aligned(z2, 16))
        return fail(CK_ERR_INVALID_ARG, "%s: expert weights, scales and zeros must be 16-byte aligned", fn);
    if (T == 0)
        return ok();
    CK_TRY(check_x(fn, x, H, ldx));
    if (routed)
        CK_TRY(check_logits(fn, logits, kind, E, ldl));
    CK_TRY(check_slots(fn, ids, weights));
    CK_TRY(check_out(fn, out, H, ldo, 2));
    const size_t need = moe_workspace(T, I, E, k);
    if (!ws || ws_bytes < need)
        return fail(CK_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, ws_bytes,
                    ws ? "" : ", NULL");
    if (!aligned(ws, kWsAlign))
        return fail(CK_ERR_WORKSPACE, "%s: workspace must be %zu-byte aligned", fn, kWsAlign);

    const Range written[] = {span(out, T, H, ldo, 2), span(ws, 1, (int64_t)need, (int64_t)need, 1),
                             span(ids, T, k, k, 4), span(weights, T, k, k, 4)};
    const Range read[] = {span(x, T, H, ldx, 2),
                          routed ? span(logits, T, E, ldl, logit_size(kind)) : Range(),
                          span(w1, E * 2 * I, H / 2, H / 2, 1),
                          span(s1, E * (H / 64), 2 * I, 2 * I, 2),
                          span(z1, E * (H / 64), 2 * I, 2 * I, 2),
                          span(w2, E * H, I / 2, I / 2, 1),
                          span(s2, E * (I / 64), H, H, 2),
                          span(z2, E * (I / 64), H, H, 2)};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlap(written[i], written[j]))
                return fail(CK_ERR_INVALID_ARG, "%s: out, workspace, ids and weights must not overlap", fn);
        if (i >= 2 && !routed)
            continue;  // given ids and weights are only read
        for (const Range &r : read)
            if (overlap(written[i], r))
                return fail(CK_ERR_INVALID_ARG, "%s: an output or the workspace overlaps an input", fn);
    }

    const ck::MoeExperts w{w1, s1, z1, w2, s2, z2, (int)E, (int)H, (int)I};
    const int64_t pass = moe_pass_tokens(T, H, k);
    for (int64_t t = 0; t < T; t += pass) {
        const int64_t n = T - t < pass ? T - t : pass;
        const ck::MoeRouting r{routed ? static_cast<const uint8_t *>(logits) + t * ldl * logit_size(kind) : nullptr,
                               kind == CK_LOGITS_BF16, renormalize != 0, ldl, k, ids + t * k, weights + t * k};
        const int e = ck::launch_moe(x + t * ldx, (int)n, ldx, r, w, out + t * ldo, ldo, ws, stream);
        if (e != 0)
            return hip_status(e, fn);
    }
    return ok();
}

size_t lora_workspace(int64_t M, int64_t K, int64_t R, int64_t L)
{
    if (M <= 0 || M > kMaxRows || K < 64 || K % 64 != 0 || K > kMaxK || R < 1 || R % 8 != 0 ||
        R > ck::kLoraMaxRank || L < 1 || L > kMaxRows)
        return 0;
    return round_up((size_t)(ck::lora_room_rows(M, K) * R) * sizeof(float), kWsAlign);
}

int ck_lora_add_impl(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, const int32_t *index, int64_t L, int64_t R,
                     const uint16_t *a, const uint16_t *b, const float *scaling, const int32_t *ranks, int64_t N,
                     const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo, void *ws, size_t ws_bytes,
                     void *stream)
{
    const char *fn = "ck_lora_add";
    CK_TRY(check_m(fn, M));
    CK_TRY(check_k(fn, K));
    if (L < 1 || R < 1 || R % 8 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: L must be positive and R a positive multiple of 8 (L=%lld, R=%lld)", fn,
                    (long long)L, (long long)R);
    if (L > kMaxRows || R > ck::kLoraMaxRank)
        return fail(CK_ERR_UNSUPPORTED, "%s: takes L <= %lld and R <= %d (L=%lld, R=%lld)", fn, (long long)kMaxRows,
                    ck::kLoraMaxRank, (long long)L, (long long)R);
    if (N <= 0)
        return fail(CK_ERR_INVALID_ARG, "%s: N must be positive (got %lld)", fn, (long long)N);
    if (N % 16 != 0 || N > kMaxRows)
        return fail(CK_ERR_UNSUPPORTED, "%s: N must be a multiple of 16 and at most %lld (got %lld)", fn,
                    (long long)kMaxRows, (long long)N);
    if (!a || !b || !aligned(a, 16) || !aligned(b, 16))
        return fail(CK_ERR_INVALID_ARG, "%s: a and b must be non-NULL 16-byte aligned pointers", fn);
    if (!aligned(scaling, 4) || !aligned(ranks, 4))
        return fail(CK_ERR_INVALID_ARG, "%s: scaling and ranks must be 4-byte aligned", fn);
    if (M == 0)
        return ok();
    CK_TRY(check_x(fn, x, K, ldx));
    if (!index || !aligned(index, 4))
        return fail(CK_ERR_INVALID_ARG, "%s: index must be a non-NULL 4-byte aligned pointer", fn);
    CK_TRY(check_out(fn, out, N, ldo, 2));
    if (base && (ldb < N || ldb % 8 != 0 || !aligned(base, 16)))
        return fail(CK_ERR_INVALID_ARG, "%s: base must be 16-byte aligned with ldb >= N, ldb %% 8 == 0", fn);
    if (ck::lora_blocks(M, N, L) >= (int64_t(1) << 24))
        return fail(CK_ERR_UNSUPPORTED, "%s: M * N too large for one launch (M=%lld, N=%lld)", fn, (long long)M,
                    (long long)N);
    const size_t need = lora_workspace(M, K, R, L);
    if (!ws || ws_bytes < need)
        return fail(CK_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, ws_bytes,
                    ws ? "" : ", NULL");
    if (!aligned(ws, kWsAlign))
        return fail(CK_ERR_WORKSPACE, "%s: workspace must be %zu-byte aligned", fn, kWsAlign);
    const Range ro = span(out, M, N, ldo, 2), rw = span(ws, 1, (int64_t)need, (int64_t)need, 1);
    const Range rb = span(base, M, N, ldb, 2);
    const Range read[] = {span(x, M, K, ldx, 2),        span(index, 1, M, M, 4),    span(a, L * R, K, K, 2),
                          span(b, L * N, R, R, 2),      span(scaling, 1, L, L, 4), span(ranks, 1, L, L, 4)};
    for (const Range &r : read)
        if (overlap(ro, r) || overlap(rw, r))
            return fail(CK_ERR_INVALID_ARG, "%s: the output or the workspace overlaps an input", fn);
    if (overlap(ro, rw) || overlap(rb, rw))
        return fail(CK_ERR_INVALID_ARG, "%s: the workspace overlaps base or out", fn);
    if (overlap(ro, rb) && !(base == out && ldb == ldo))
        return fail(CK_ERR_INVALID_ARG, "%s: base overlaps out and is not out itself", fn);
    return hip_status(ck::launch_lora(x, M, (int)K, ldx, index, L, (int)R, a, b, scaling, ranks, (int)N, base, ldb,
                                      out, ldo, static_cast<float *>(ws), stream),
                      fn);
}

}  // namespace

extern "C" {

ck_status ck_moe_route(const void *logits, int32_t logit_kind, int64_t T, int64_t E, int64_t ldl, int32_t k,
                       int32_t renormalize, int32_t *ids, float *weights, void *stream)
{
    return static_cast<ck_status>(
        ck_moe_route_impl(logits, logit_kind, T, E, ldl, k, renormalize, ids, weights, stream));
}

size_t ck_moe_workspace_bytes(int64_t T, int64_t I, int64_t E, int32_t k) { return moe_workspace(T, I, E, k); }

ck_status ck_moe_w4a16(const uint16_t *x, int64_t T, int64_t H, int64_t ldx, const void *logits, int32_t logit_kind,
                       int64_t ldl, int32_t k, int32_t renormalize, int64_t E, int64_t I, int32_t Gw,
                       const uint8_t *w1, const uint16_t *s1, const uint16_t *z1, const uint8_t *w2,
                       const uint16_t *s2, const uint16_t *z2, uint16_t *out, int64_t ldo, int32_t *ids,
                       float *weights, void *ws, size_t ws_bytes, void *stream)
{
    return static_cast<ck_status>(moe_common("ck_moe_w4a16", x, T, H, ldx, logits, logit_kind, ldl, renormalize, true,
                                             ids, weights, k, E, I, Gw, w1, s1, z1, w2, s2, z2, out, ldo, ws,
                                             ws_bytes, stream));
}

ck_status ck_moe_experts_w4a16(const uint16_t *x, int64_t T, int64_t H, int64_t ldx, const int32_t *ids,
                               const float *weights, int32_t k, int64_t E, int64_t I, int32_t Gw, const uint8_t *w1,
                               const uint16_t *s1, const uint16_t *z1, const uint8_t *w2, const uint16_t *s2,
                               const uint16_t *z2, uint16_t *out, int64_t ldo, void *ws, size_t ws_bytes,
                               void *stream)
{
    return static_cast<ck_status>(moe_common("ck_moe_experts_w4a16", x, T, H, ldx, nullptr, CK_LOGITS_F32, E, 0, false,
                                             const_cast<int32_t *>(ids), const_cast<float *>(weights), k, E, I, Gw,
                                             w1, s1, z1, w2, s2, z2, out, ldo, ws, ws_bytes, stream));
}

size_t ck_lora_workspace_bytes(int64_t M, int64_t K, int64_t R, int64_t L) { return lora_workspace(M, K, R, L); }

ck_status ck_lora_add(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, const int32_t *index, int64_t L,
                      int64_t R, const uint16_t *a, const uint16_t *b, const float *scaling, const int32_t *ranks,
                      int64_t N, const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo, void *ws,
                      size_t ws_bytes, void *stream)
{
    return static_cast<ck_status>(ck_lora_add_impl(x, M, K, ldx, index, L, R, a, b, scaling, ranks, N, base, ldb, out,
                                                   ldo, ws, ws_bytes, stream));
}

}  // extern "C"
