// C ABI of the 8-bit float operators: quantisers, linears with a scale for each block of
// 128, the gated feed-forward block and its backward pass.  Validation and dispatch as
// in ck_api.cpp: nothing is enqueued until every check has passed.  Semantics are
// documented in include/ck.h.
#include "../../include/ck.h"

#include "api_check.h"
#include "fp8_launch.h"

namespace {

using namespace ck::api;

// Row strides in bytes: a tile's 256 rows are addressed with 32-bit buffer offsets.
constexpr int64_t kMaxLd = int64_t(1) << 23;

int check_columns(const char *fn, const char *name, int64_t K, int64_t of = 16)
{
    if (K <= 0 || K % of != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: %s must be a positive multiple of %lld (got %lld)", fn, name,
                    (long long)of, (long long)K);
    if (K > kMaxK)
        return fail(CK_ERR_UNSUPPORTED, "%s: %s must be at most %lld (got %lld)", fn, name, (long long)kMaxK,
                    (long long)K);
    return CK_OK;
}

int check_rows(const char *fn, int64_t N)
{
    if (N <= 0)
        return fail(CK_ERR_INVALID_ARG, "%s: N must be positive (got %lld)", fn, (long long)N);
    if (N % 16 != 0 || N > kMaxRows)
        return fail(CK_ERR_UNSUPPORTED, "%s: N must be a multiple of 16 and at most %lld (got %lld)", fn,
                    (long long)kMaxRows, (long long)N);
    return CK_OK;
}

int check_codes(const char *fn, const char *name, const uint8_t *codes, int64_t K, int64_t ld)
{
    if (!codes || !aligned(codes, 16))
        return fail(CK_ERR_INVALID_ARG, "%s: %s must be a non-NULL 16-byte aligned pointer", fn, name);
    if (ld < K || ld % 16 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: the row stride of %s (%lld) must be >= %lld and a multiple of 16", fn,
                    name, (long long)ld, (long long)K);
    if (ld > kMaxLd)
        return fail(CK_ERR_UNSUPPORTED, "%s: the row stride of %s (%lld) must be at most %lld bytes", fn, name,
                    (long long)ld, (long long)kMaxLd);
    return CK_OK;
}

int check_scales(const char *fn, const uint8_t *scales, int64_t K, int64_t lds)
{
    if (!scales || !aligned(scales, 4))
        return fail(CK_ERR_INVALID_ARG, "%s: scales must be a non-NULL 4-byte aligned pointer", fn);
    if (lds < ck::fp8_blocks(K) || lds % 4 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: lds (%lld) must be >= ceil(K / 128) and a multiple of 4", fn,
                    (long long)lds);
    if (lds > kMaxLd)
        return fail(CK_ERR_UNSUPPORTED, "%s: lds (%lld) must be at most %lld", fn, (long long)lds, (long long)kMaxLd);
    return CK_OK;
}

int check_weight_scales(const char *fn, const char *name, const uint8_t *scales)
{
    if (!scales)
        return fail(CK_ERR_INVALID_ARG, "%s: %s must not be NULL", fn, name);
    return CK_OK;
}

int check_tiles(const char *fn, int64_t M, int64_t N)
{
    if (ck::fp8_tiles(M, N) > ck::kFp8MaxTiles)
        return fail(CK_ERR_UNSUPPORTED, "%s: M * N too large for one launch (M=%lld, N=%lld)", fn, (long long)M,
                    (long long)N);
    return CK_OK;
}

int check_space(const char *fn, const void *ws, size_t ws_bytes, size_t need)
{
    if (!ws || ws_bytes < need)
        return fail(CK_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, ws_bytes,
                    ws ? "" : ", NULL");
    if (!aligned(ws, kWsAlign))
        return fail(CK_ERR_WORKSPACE, "%s: workspace must be %zu-byte aligned", fn, kWsAlign);
    return CK_OK;
}

// No two written ranges overlap, and none overlaps a read one.
template <size_t W, size_t R>
int check_apart(const char *fn, const Range (&written)[W], const Range (&read)[R])
{
    for (size_t i = 0; i < W; ++i) {
        for (size_t j = i + 1; j < W; ++j)
            if (overlap(written[i], written[j]))
                return fail(CK_ERR_INVALID_ARG, "%s: the outputs and the workspace must not overlap", fn);
        for (const Range &r : read)
            if (overlap(written[i], r))
                return fail(CK_ERR_INVALID_ARG, "%s: an output or the workspace overlaps an input", fn);
    }
    return CK_OK;
}

Range codes_span(const uint8_t *p, int64_t M, int64_t K, int64_t ld) { return span(p, M, K, ld, 1); }
// Rows of scales up to the next multiple of four bytes.
Range scales_span(const uint8_t *p, int64_t M, int64_t K, int64_t lds)
{
    return span(p, M, ck::fp8_scale_stride(K), lds, 1);
}
Range weight_scales_span(const uint8_t *p, int64_t N, int64_t K)
{
    return span(p, ck::fp8_blocks(N), ck::fp8_blocks(K), ck::fp8_blocks(K), 1);
}

// Quantised activations [M, K] inside a workspace.
size_t codes_bytes(int64_t M, int64_t K) { return round_up((size_t)M * (size_t)K, kWsAlign); }
size_t scales_bytes(int64_t M, int64_t K) { return round_up((size_t)(M * ck::fp8_scale_stride(K)), kWsAlign); }
size_t quantised_bytes(int64_t M, int64_t K) { return codes_bytes(M, K) + scales_bytes(M, K); }

struct Quantised {
    uint8_t *codes, *scales;
    int64_t stride;
};
Quantised take(uint8_t *&at, int64_t M, int64_t K)
{
    const Quantised q{at, at + codes_bytes(M, K), ck::fp8_scale_stride(K)};
    at += quantised_bytes(M, K);
    return q;
}

bool serves(int64_t M, int64_t K, int64_t of) { return M > 0 && M <= kMaxRows && K > 0 && K % of == 0 && K <= kMaxK; }

size_t linear_bytes(int64_t M, int64_t K, int64_t N)
{
    return serves(M, K, 16) && N > 0 && N % 16 == 0 && N <= kMaxRows
               ? quantised_bytes(M, K) + round_up((size_t)ck::fp8_split_floats(M, K, N) * sizeof(float), kWsAlign)
               : 0;
}
// fp32 results of the few-row products, between a block's two; then the sums of the second, where
// it is split.
size_t sums_bytes(int64_t M, int64_t H, int64_t I)
{
    const int64_t few = (M < ck::kFp8FewRows ? M : ck::kFp8FewRows) * I, split = ck::fp8_split_floats(M, I, H);
    return round_up((size_t)(few > split ? few : split) * sizeof(float), kWsAlign);
}
// x, what lies between the two products, and its fp32 form.
size_t pair_bytes(int64_t M, int64_t H, int64_t inner)
{
    return quantised_bytes(M, H) + quantised_bytes(M, inner) + sums_bytes(M, H, inner);
}
size_t ffn_bytes(int64_t M, int64_t H, int64_t I)
{
    return serves(M, H, 16) && serves(M, I, 128) ? pair_bytes(M, H, I) : 0;
}
size_t backward_bytes(int64_t M, int64_t H, int64_t I)
{
    return serves(M, H, 16) && serves(M, I, 128) ? pair_bytes(M, H, 2 * I) : 0;
}

// A product on the kernel that takes the least time.  sums: room for the few-row product's fp32
// results and for a split product's, or null.
struct Choice {
    ck::Fp8Plan plan;
    bool few;
};
Choice choose(ck::Fp8Result kind, const ck::Fp8Product &p, bool room)
{
    const int64_t cols = kind == ck::Fp8Result::kBf16 ? p.N : p.I;
    const ck::Fp8Plan plan = ck::fp8_plan(kind, p.M, p.K, cols, room);
    return {plan, ck::fp8_few(kind, p.M, p.K, cols, plan)};
}
int from_codes(ck::Fp8Result kind, const ck::Fp8Product &p, float *sums, void *stream)
{
    const Choice c = choose(kind, p, sums != nullptr);
    return c.few ? ck::launch_fp8_few(kind, p, nullptr, false, 0, sums, stream)
                 : ck::launch_fp8_tiled(kind, p, c.plan, sums, stream);
}

// A product of bf16 (or fp32) rows: quantised on the way where that pays, through q otherwise.
int from_rows(ck::Fp8Result kind, ck::Fp8Product &p, const void *x, bool f32, int64_t ldx, const Quantised &q,
              float *sums, void *stream)
{
    if (ck::fp8_few_raw(p.M, p.K))
        return ck::launch_fp8_few(kind, p, x, f32, ldx, sums, stream);
    const int e = ck::launch_fp8_quant(x, f32, p.M, p.K, ldx, q.codes, p.K, q.scales, q.stride, stream);
    if (e != 0)
        return e;
    p.a = q.codes, p.lda = p.K, p.sa = q.scales, p.ldsa = q.stride;
    return from_codes(kind, p, sums, stream);
}

// The two products of a feed-forward block, or of its backward pass.
int two_products(ck::Fp8Result kind, ck::Fp8Product &first, ck::Fp8Product &second, const uint16_t *x, int64_t ldx,
                 void *ws, void *stream)
{
    uint8_t *at = static_cast<uint8_t *>(ws);
    const Quantised q = take(at, first.M, first.K), h = take(at, first.M, second.K);
    float *sums = reinterpret_cast<float *>(at);
    first.q = h.codes, first.sq = h.scales, first.ldsq = h.stride;
    const int e = from_rows(kind, first, x, false, ldx, q, sums, stream);
    if (e != 0)
        return e;
    if (ck::fp8_few_raw(first.M, first.K) || choose(kind, first, true).few)
        return from_rows(ck::Fp8Result::kBf16, second, sums, true, second.K, h, sums, stream);
    second.a = h.codes, second.lda = second.K, second.sa = h.scales, second.ldsa = h.stride;
    return from_codes(ck::Fp8Result::kBf16, second, sums, stream);
}

int quant_impl(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, uint8_t *codes, int64_t ldq, uint8_t *scales,
               int64_t lds, void *stream)
{
    const char *fn = "ck_fp8_quant";
    CK_TRY(check_m(fn, M));
    CK_TRY(check_columns(fn, "K", K));
    if (M == 0)
        return ok();
    CK_TRY(check_x(fn, x, K, ldx));
    CK_TRY(check_codes(fn, "codes", codes, K, ldq));
    CK_TRY(check_scales(fn, scales, K, lds));
    CK_TRY(check_apart(fn, {codes_span(codes, M, K, ldq), span(scales, M, ck::fp8_blocks(K), lds, 1)},
                       {span(x, M, K, ldx, 2)}));
    return hip_status(ck::launch_fp8_quant(x, false, M, (int)K, ldx, codes, ldq, scales, lds, stream), fn);
}

int quantize_weights_impl(const uint16_t *w, int64_t N, int64_t K, int64_t ldw_in, uint8_t *codes, int64_t ldw,
                          uint8_t *scales, void *stream)
{
    const char *fn = "ck_fp8_quantize_weights";
    CK_TRY(check_columns(fn, "K", K));
    CK_TRY(check_rows(fn, N));
    if (!w || !aligned(w, 16) || ldw_in < K || ldw_in % 8 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: w must be 16-byte aligned with ldw_in >= K, ldw_in %% 8 == 0", fn);
    CK_TRY(check_codes(fn, "codes", codes, K, ldw));
    CK_TRY(check_weight_scales(fn, "scales", scales));
    CK_TRY(check_apart(fn, {codes_span(codes, N, K, ldw), weight_scales_span(scales, N, K)},
                       {span(w, N, K, ldw_in, 2)}));
    return hip_status(ck::launch_fp8_quantize_weights(w, N, (int)K, ldw_in, codes, ldw, scales, stream), fn);
}

int transpose_impl(const uint8_t *codes, int64_t ldw, const uint8_t *scales, int64_t N, int64_t K, uint8_t *codes_t,
                   int64_t ldt, uint8_t *scales_t, void *stream)
{
    const char *fn = "ck_fp8_transpose_weights";
    // Either may be a linear's outputs, so neither is held to the limit of a product's columns.
    CK_TRY(check_rows(fn, N));
    CK_TRY(check_rows(fn, K));
    CK_TRY(check_codes(fn, "codes", codes, K, ldw));
    CK_TRY(check_codes(fn, "codes_t", codes_t, N, ldt));
    CK_TRY(check_weight_scales(fn, "scales", scales));
    CK_TRY(check_weight_scales(fn, "scales_t", scales_t));
    CK_TRY(check_apart(fn, {codes_span(codes_t, K, N, ldt), weight_scales_span(scales_t, K, N)},
                       {codes_span(codes, N, K, ldw), weight_scales_span(scales, N, K)}));
    return hip_status(ck::launch_fp8_transpose(codes, ldw, scales, (int)N, (int)K, codes_t, ldt, scales_t, stream),
                      fn);
}

// The checks of a linear's weight, bias and result.
int check_linear(const char *fn, int64_t M, int64_t K, const uint8_t *w, int64_t ldw, const uint8_t *w_scales,
                 int64_t N, const uint16_t *bias, uint16_t *out, int64_t ldo)
{
    CK_TRY(check_codes(fn, "w", w, K, ldw));
    CK_TRY(check_weight_scales(fn, "w_scales", w_scales));
    if (!aligned(bias, 2))
        return fail(CK_ERR_INVALID_ARG, "%s: bias must be 2-byte aligned", fn);
    if (M == 0)
        return CK_OK;
    CK_TRY(check_out(fn, out, N, ldo, 2));
    return check_tiles(fn, M, N);
}

ck::Fp8Product product(int64_t M, int64_t K, const uint8_t *w, int64_t ldw, const uint8_t *sw, int64_t N)
{
    ck::Fp8Product p{};
    p.M = M, p.K = (int)K, p.w = w, p.ldw = ldw, p.sw = sw, p.N = (int)N;
    return p;
}

int gemm_impl(const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds, int64_t M, int64_t K,
              const uint8_t *w, int64_t ldw, const uint8_t *w_scales, int64_t N, const uint16_t *bias, uint16_t *out,
              int64_t ldo, void *stream)
{
    const char *fn = "ck_fp8_gemm";
    CK_TRY(check_m(fn, M));
    CK_TRY(check_columns(fn, "K", K));
    CK_TRY(check_rows(fn, N));
    CK_TRY(check_linear(fn, M, K, w, ldw, w_scales, N, bias, out, ldo));
    if (M == 0)
        return ok();
    CK_TRY(check_codes(fn, "codes", codes, K, ldq));
    CK_TRY(check_scales(fn, scales, K, lds));
    CK_TRY(check_apart(fn, {span(out, M, N, ldo, 2)},
                       {codes_span(codes, M, K, ldq), scales_span(scales, M, K, lds), codes_span(w, N, K, ldw),
                        weight_scales_span(w_scales, N, K), span(bias, 1, N, N, 2)}));
    ck::Fp8Product p = product(M, K, w, ldw, w_scales, N);
    p.a = codes, p.lda = ldq, p.sa = scales, p.ldsa = lds;
    p.bias = bias, p.out = out, p.ldo = ldo;
    return hip_status(from_codes(ck::Fp8Result::kBf16, p, nullptr, stream), fn);
}

int linear_impl(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, const uint8_t *w, int64_t ldw,
                const uint8_t *w_scales, int64_t N, const uint16_t *bias, uint16_t *out, int64_t ldo, void *ws,
                size_t ws_bytes, void *stream)
{
    const char *fn = "ck_fp8_linear";
    CK_TRY(check_m(fn, M));
    CK_TRY(check_columns(fn, "K", K));
    CK_TRY(check_rows(fn, N));
    CK_TRY(check_linear(fn, M, K, w, ldw, w_scales, N, bias, out, ldo));
    if (M == 0)
        return ok();
    CK_TRY(check_x(fn, x, K, ldx));
    const size_t need = linear_bytes(M, K, N);
    CK_TRY(check_space(fn, ws, ws_bytes, need));
    CK_TRY(check_apart(fn, {span(out, M, N, ldo, 2), span(ws, 1, (int64_t)need, (int64_t)need, 1)},
                       {span(x, M, K, ldx, 2), codes_span(w, N, K, ldw), weight_scales_span(w_scales, N, K),
                        span(bias, 1, N, N, 2)}));
    uint8_t *at = static_cast<uint8_t *>(ws);
    const Quantised q = take(at, M, K);
    ck::Fp8Product p = product(M, K, w, ldw, w_scales, N);
    p.bias = bias, p.out = out, p.ldo = ldo;
    return hip_status(from_rows(ck::Fp8Result::kBf16, p, x, false, ldx, q, reinterpret_cast<float *>(at), stream), fn);
}

int check_ffn(const char *fn, int64_t M, int64_t H, int64_t I, const uint8_t *w1, const uint8_t *s1, const uint8_t *w2,
              const uint8_t *s2)
{
    CK_TRY(check_m(fn, M));
    CK_TRY(check_columns(fn, "H", H));
    CK_TRY(check_columns(fn, "I", I, 128));
    CK_TRY(check_codes(fn, "the first weight", w1, 16, 16));
    CK_TRY(check_codes(fn, "the second weight", w2, 16, 16));
    CK_TRY(check_weight_scales(fn, "the first weight's scales", s1));
    return check_weight_scales(fn, "the second weight's scales", s2);
}

int check_gate_up(const char *fn, const uint16_t *gate_up, int64_t I, int64_t ldg)
{
    if (!gate_up || !aligned(gate_up, 16) || ldg < 2 * I || ldg % 8 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s: gate_up must be 16-byte aligned with ldg >= 2 I, ldg %% 8 == 0", fn);
    return CK_OK;
}

int ffn_impl(const uint16_t *x, int64_t M, int64_t H, int64_t ldx, int64_t I, const uint8_t *w1, const uint8_t *s1,
             const uint8_t *w2, const uint8_t *s2, uint16_t *out, int64_t ldo, uint16_t *gate_up, int64_t ldg,
             void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "ck_fp8_ffn";
    CK_TRY(check_ffn(fn, M, H, I, w1, s1, w2, s2));
    if (M == 0)
        return ok();
    CK_TRY(check_x(fn, x, H, ldx));
    CK_TRY(check_out(fn, out, H, ldo, 2));
    if (gate_up)
        CK_TRY(check_gate_up(fn, gate_up, I, ldg));
    CK_TRY(check_tiles(fn, M, 2 * I));
    CK_TRY(check_tiles(fn, M, H));
    const size_t need = ffn_bytes(M, H, I);
    CK_TRY(check_space(fn, ws, ws_bytes, need));
    CK_TRY(check_apart(fn,
                       {span(out, M, H, ldo, 2), span(gate_up, M, 2 * I, ldg, 2),
                        span(ws, 1, (int64_t)need, (int64_t)need, 1)},
                       {span(x, M, H, ldx, 2), codes_span(w1, 2 * I, H, H), weight_scales_span(s1, 2 * I, H),
                        codes_span(w2, H, I, I), weight_scales_span(s2, H, I)}));
    ck::Fp8Product first = product(M, H, w1, H, s1, 2 * I), second = product(M, I, w2, I, s2, H);
    first.I = (int)I, first.gate_up = gate_up, first.ldg = ldg;
    second.out = out, second.ldo = ldo;
    return hip_status(two_products(ck::Fp8Result::kGated, first, second, x, ldx, ws, stream), fn);
}

int backward_impl(const uint16_t *dy, int64_t M, int64_t H, int64_t ldy, const uint16_t *gate_up, int64_t ldg,
                  int64_t I, const uint8_t *w1t, const uint8_t *s1t, const uint8_t *w2t, const uint8_t *s2t,
                  uint16_t *dx, int64_t lddx, void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "ck_fp8_ffn_backward";
    CK_TRY(check_ffn(fn, M, H, I, w1t, s1t, w2t, s2t));
    if (M == 0)
        return ok();
    CK_TRY(check_x(fn, dy, H, ldy));
    CK_TRY(check_gate_up(fn, gate_up, I, ldg));
    CK_TRY(check_out(fn, dx, H, lddx, 2));
    CK_TRY(check_tiles(fn, M, I));
    CK_TRY(check_tiles(fn, M, H));
    const size_t need = backward_bytes(M, H, I);
    CK_TRY(check_space(fn, ws, ws_bytes, need));
    CK_TRY(check_apart(fn, {span(dx, M, H, lddx, 2), span(ws, 1, (int64_t)need, (int64_t)need, 1)},
                       {span(dy, M, H, ldy, 2), span(gate_up, M, 2 * I, ldg, 2), codes_span(w1t, H, 2 * I, 2 * I),
                        weight_scales_span(s1t, H, 2 * I), codes_span(w2t, I, H, H), weight_scales_span(s2t, I, H)}));
    ck::Fp8Product first = product(M, H, w2t, H, s2t, I), second = product(M, 2 * I, w1t, 2 * I, s1t, H);
    first.I = (int)I, first.gate_up = const_cast<uint16_t *>(gate_up), first.ldg = ldg;
    second.out = dx, second.ldo = lddx;
    return hip_status(two_products(ck::Fp8Result::kGrad, first, second, dy, ldy, ws, stream), fn);
}

}  // namespace

extern "C" {

ck_status ck_fp8_quant(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, uint8_t *codes, int64_t ldq,
                       uint8_t *scales, int64_t lds, void *stream)
{
    return static_cast<ck_status>(quant_impl(x, M, K, ldx, codes, ldq, scales, lds, stream));
}

ck_status ck_fp8_quantize_weights(const uint16_t *w, int64_t N, int64_t K, int64_t ldw_in, uint8_t *codes,
                                  int64_t ldw, uint8_t *scales, void *stream)
{
    return static_cast<ck_status>(quantize_weights_impl(w, N, K, ldw_in, codes, ldw, scales, stream));
}

ck_status ck_fp8_transpose_weights(const uint8_t *codes, int64_t ldw, const uint8_t *scales, int64_t N, int64_t K,
                                   uint8_t *codes_t, int64_t ldt, uint8_t *scales_t, void *stream)
{
    return static_cast<ck_status>(transpose_impl(codes, ldw, scales, N, K, codes_t, ldt, scales_t, stream));
}

ck_status ck_fp8_gemm(const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds, int64_t M, int64_t K,
                      const uint8_t *w, int64_t ldw, const uint8_t *w_scales, int64_t N, const uint16_t *bias,
                      uint16_t *out, int64_t ldo, void *stream)
{
    return static_cast<ck_status>(
        gemm_impl(codes, ldq, scales, lds, M, K, w, ldw, w_scales, N, bias, out, ldo, stream));
}

size_t ck_fp8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N) { return linear_bytes(M, K, N); }

ck_status ck_fp8_linear(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, const uint8_t *w, int64_t ldw,
                        const uint8_t *w_scales, int64_t N, const uint16_t *bias, uint16_t *out, int64_t ldo,
                        void *ws, size_t ws_bytes, void *stream)
{
    return static_cast<ck_status>(
        linear_impl(x, M, K, ldx, w, ldw, w_scales, N, bias, out, ldo, ws, ws_bytes, stream));
}

size_t ck_fp8_ffn_workspace_bytes(int64_t M, int64_t H, int64_t I) { return ffn_bytes(M, H, I); }
size_t ck_fp8_ffn_backward_workspace_bytes(int64_t M, int64_t H, int64_t I) { return backward_bytes(M, H, I); }

ck_status ck_fp8_ffn(const uint16_t *x, int64_t M, int64_t H, int64_t ldx, int64_t I, const uint8_t *w1,
                     const uint8_t *s1, const uint8_t *w2, const uint8_t *s2, uint16_t *out, int64_t ldo,
                     uint16_t *gate_up, int64_t ldg, void *ws, size_t ws_bytes, void *stream)
{
    return static_cast<ck_status>(
        ffn_impl(x, M, H, ldx, I, w1, s1, w2, s2, out, ldo, gate_up, ldg, ws, ws_bytes, stream));
}

ck_status ck_fp8_ffn_backward(const uint16_t *dy, int64_t M, int64_t H, int64_t ldy, const uint16_t *gate_up,
                              int64_t ldg, int64_t I, const uint8_t *w1t, const uint8_t *s1t, const uint8_t *w2t,
                              const uint8_t *s2t, uint16_t *dx, int64_t lddx, void *ws, size_t ws_bytes, void *stream)
{
    return static_cast<ck_status>(backward_impl(dy, M, H, ldy, gate_up, ldg, I, w1t, s1t, w2t, s2t, dx, lddx, ws,
                                                ws_bytes, stream));
}

}  // extern "C"
