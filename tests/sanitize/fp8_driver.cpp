// Drives the entry points of ck_fp8_api.cpp against host stand-ins for their launchers,
// under AddressSanitizer and UndefinedBehaviorSanitizer.  The stand-ins touch the first
// and the last byte of everything the kernels may reach, in buffers of exactly the
// documented sizes, and check what a launcher may rely on.
// Prints "fp8 driver: N checks, 0 failures" and exits 0 when all pass.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>
#include <vector>

#include "../../include/ck.h"
#include "../../packed_int4_convrot_amd/csrc/fp8_launch.h"

namespace {

int g_checks = 0, g_failures = 0;

#define EXPECT(cond)                                                               \
    do {                                                                           \
        ++g_checks;                                                                \
        if (!(cond)) {                                                             \
            ++g_failures;                                                          \
            fprintf(stderr, "%s:%d: EXPECT(%s) failed; last error: %s\n", __FILE__, \
                    __LINE__, #cond, ck_last_error_msg());                         \
        }                                                                          \
    } while (0)

// Buffers of an exact size, 256-byte aligned.
struct Pool {
    std::vector<void *> all;
    template <class T>
    T *get(int64_t bytes)
    {
        void *p = nullptr;
        if (posix_memalign(&p, 256, bytes > 0 ? (size_t)bytes : 1) != 0)
            exit(2);
        all.push_back(p);
        return static_cast<T *>(p);
    }
    ~Pool()
    {
        for (void *p : all)
            free(p);
    }
};

volatile uint8_t g_sink;

void read_span(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t esize)
{
    if (!p || rows <= 0)
        return;
    const uint8_t *b = static_cast<const uint8_t *>(p);
    g_sink = b[0];
    g_sink = b[((rows - 1) * ld + cols) * esize - 1];
}
void write_span(void *p, int64_t rows, int64_t cols, int64_t ld, int64_t esize)
{
    if (!p || rows <= 0)
        return;
    uint8_t *b = static_cast<uint8_t *>(p);
    b[0] = 1;
    b[((rows - 1) * ld + cols) * esize - 1] = 1;
}

int g_calls, g_fail_at;   // launches, and the one that fails (0: none)

int finish()
{
    return ++g_calls == g_fail_at ? 7 : 0;
}

void touch_product(ck::Fp8Result kind, const ck::Fp8Product &p)
{
    const int64_t steps = ck::fp8_blocks(p.K);
    EXPECT(p.M > 0 && p.K % 16 == 0 && p.N % 16 == 0 && p.ldw % 16 == 0);
    read_span(p.w, p.N, p.K, p.ldw, 1);
    read_span(p.sw, ck::fp8_blocks(p.N), steps, steps, 1);
    if (kind == ck::Fp8Result::kBf16) {
        read_span(p.bias, 1, p.N, p.N, 2);
        write_span(p.out, p.M, p.N, p.ldo, 2);
    } else {
        EXPECT(p.I % 128 == 0 && p.N == (kind == ck::Fp8Result::kGated ? 2 * p.I : p.I));
        if (kind == ck::Fp8Result::kGated)
            write_span(p.gate_up, p.M, 2 * p.I, p.ldg, 2);
        else
            read_span(p.gate_up, p.M, 2 * p.I, p.ldg, 2);
    }
}
void touch_rows(const ck::Fp8Product &p)
{
    EXPECT(p.a && p.sa && p.lda % 16 == 0 && p.ldsa % 4 == 0);
    read_span(p.a, p.M, p.K, p.lda, 1);
    read_span(p.sa, p.M, ck::fp8_scale_stride(p.K), p.ldsa, 1);
}
int64_t inner(ck::Fp8Result kind, const ck::Fp8Product &p) { return kind == ck::Fp8Result::kGrad ? 2 * (int64_t)p.I : p.I; }

}  // namespace

namespace ck {

int launch_fp8_quant(const void *x, bool f32, int64_t M, int K, int64_t ldx, uint8_t *codes, int64_t lda,
                     uint8_t *scales, int64_t ldsa, void *)
{
    read_span(x, M, K, ldx, f32 ? 4 : 2);
    write_span(codes, M, K, lda, 1);
    write_span(scales, M, fp8_blocks(K), ldsa, 1);
    return finish();
}

int launch_fp8_quantize_weights(const uint16_t *w, int64_t N, int K, int64_t ldw_in, uint8_t *codes, int64_t ldw,
                                uint8_t *scales, void *)
{
    read_span(w, N, K, ldw_in, 2);
    write_span(codes, N, K, ldw, 1);
    write_span(scales, fp8_blocks(N), fp8_blocks(K), fp8_blocks(K), 1);
    return finish();
}

int launch_fp8_transpose(const uint8_t *codes, int64_t ldw, const uint8_t *scales, int N, int K, uint8_t *codes_t,
                         int64_t ldt, uint8_t *scales_t, void *)
{
    read_span(codes, N, K, ldw, 1);
    read_span(scales, fp8_blocks(N), fp8_blocks(K), fp8_blocks(K), 1);
    write_span(codes_t, K, N, ldt, 1);
    write_span(scales_t, fp8_blocks(K), fp8_blocks(N), fp8_blocks(N), 1);
    return finish();
}

int launch_fp8_tiled(Fp8Result kind, const Fp8Product &p, const Fp8Plan &plan, float *sums, void *)
{
    if (plan.splits > 1) {   // a tile's sums are written whole
        EXPECT(kind == Fp8Result::kBf16 && sums != nullptr && plan.splits <= kFp8MostSplits && plan.each % 4 == 0);
        EXPECT((plan.splits - 1) * plan.each < fp8_blocks(p.K) && plan.splits * plan.each >= fp8_blocks(p.K));
        EXPECT(plan.tile == Fp8Tile::k128x128 || plan.tile == Fp8Tile::k128x64 || plan.tile == Fp8Tile::k64x64);
        const int64_t n = plan.tile == Fp8Tile::k64x64 ? 64 : 128, m = plan.tile == Fp8Tile::k128x128 ? 128 : 64;
        const int64_t floats = plan.splits * ((p.N + n - 1) / n * n) * ((p.M + m - 1) / m * m);
        EXPECT(floats <= fp8_split_floats(p.M, p.K, p.N));
        write_span(sums, 1, floats, floats, 4);
    }
    touch_product(kind, p);
    touch_rows(p);
    if (kind != Fp8Result::kBf16) {
        write_span(p.q, p.M, inner(kind, p), inner(kind, p), 1);
        write_span(p.sq, p.M, fp8_blocks(inner(kind, p)), p.ldsq, 1);
    }
    return finish();
}

int launch_fp8_few(Fp8Result kind, const Fp8Product &p, const void *x, bool f32, int64_t ldx, float *sums, void *)
{
    const int64_t columns = kind == Fp8Result::kBf16 ? p.N : p.I;
    EXPECT(x || columns <= fp8_few_columns(kind, (p.M + 15) / 16));
    EXPECT(p.M <= kFp8FewRows && p.M * fp8_scale_stride(p.K) <= 16 * 1024);
    touch_product(kind, p);
    if (x) {
        EXPECT(fp8_few_raw(p.M, p.K));
        read_span(x, p.M, p.K, ldx, f32 ? 4 : 2);
    } else {
        touch_rows(p);
    }
    if (kind != Fp8Result::kBf16) {
        EXPECT(sums != nullptr);
        write_span(sums, p.M, inner(kind, p), inner(kind, p), 4);
    }
    return finish();
}

}  // namespace ck

namespace {

// A call that succeeds, and the same with each of its launches failing.
template <class F>
void runs(F call)
{
    g_fail_at = 0, g_calls = 0;
    EXPECT(call() == CK_OK && g_calls >= 1);
    EXPECT(ck_last_error_msg()[0] == 0);
    for (int n = g_calls; n >= 1; --n) {
        g_fail_at = n, g_calls = 0;
        EXPECT(call() == CK_ERR_HIP && g_calls == n);
        EXPECT(ck_last_error_msg()[0] != 0);
    }
    g_fail_at = 0;
}

void linears()
{
    const struct {
        int64_t M, K, N, pad;
    } cases[] = {{1, 16, 16, 0},       {3, 144, 48, 16},     {8, 2048, 128, 0},   {9, 2048, 144, 16},  {1, 32768, 16, 0},
                 {64, 32768, 32, 0},   {63, 400, 1040, 16},  {65, 128, 256, 0},   {300, 2112, 48, 32}, {5000, 16, 4096, 0}};
    for (const auto &c : cases)
        for (bool biased : {true, false}) {
            Pool p;
            const int64_t ldx = c.K + c.pad, ldw = c.K + c.pad, ldo = c.N + c.pad;
            const int64_t blocks = ck::fp8_blocks(c.K), lds = ck::fp8_scale_stride(c.K) + (c.pad ? 4 : 0);
            uint16_t *x = p.get<uint16_t>(((c.M - 1) * ldx + c.K) * 2);
            uint8_t *w = p.get<uint8_t>((c.N - 1) * ldw + c.K), *sw = p.get<uint8_t>(ck::fp8_blocks(c.N) * blocks);
            uint16_t *bias = biased ? p.get<uint16_t>(c.N * 2) : nullptr;
            uint16_t *out = p.get<uint16_t>(((c.M - 1) * ldo + c.N) * 2);
            uint8_t *codes = p.get<uint8_t>((c.M - 1) * ldw + c.K);
            uint8_t *scales = p.get<uint8_t>((c.M - 1) * lds + ck::fp8_scale_stride(c.K));
            const size_t need = ck_fp8_linear_workspace_bytes(c.M, c.K, c.N);
            uint8_t *ws = p.get<uint8_t>((int64_t)need);
            EXPECT(need > 0 && need % 256 == 0);
            const auto linear = [&](size_t bytes) {
                return ck_fp8_linear(x, c.M, c.K, ldx, w, ldw, sw, c.N, bias, out, ldo, ws, bytes, nullptr);
            };
            runs([&] { return linear(need); });
            g_calls = 0;
            EXPECT(linear(need - 1) == CK_ERR_WORKSPACE && g_calls == 0);
            runs([&] { return ck_fp8_quant(x, c.M, c.K, ldx, codes, ldw, scales, lds, nullptr); });
            runs([&] {
                return ck_fp8_gemm(codes, ldw, scales, lds, c.M, c.K, w, ldw, sw, c.N, bias, out, ldo, nullptr);
            });
            uint16_t *wide = p.get<uint16_t>(((c.N - 1) * ldw + c.K) * 2);
            runs([&] { return ck_fp8_quantize_weights(wide, c.N, c.K, ldw, w, ldw, sw, nullptr); });
            const int64_t ldt = c.N + c.pad;
            uint8_t *wt = p.get<uint8_t>((c.K - 1) * ldt + c.N), *st = p.get<uint8_t>(blocks * ck::fp8_blocks(c.N));
            runs([&] { return ck_fp8_transpose_weights(w, ldw, sw, c.N, c.K, wt, ldt, st, nullptr); });
        }
}

void blocks()
{
    const struct {
        int64_t M, H, I, pad;
    } cases[] = {{1, 16, 128, 0},   {1, 3840, 10240, 0}, {4, 144, 256, 8},   {8, 2048, 128, 0},  {9, 400, 384, 8},
                 {64, 64, 32768, 0}, {64, 32768, 128, 0}, {65, 144, 128, 16}, {700, 272, 256, 0}};
    for (const auto &c : cases)
        for (bool keep : {true, false}) {
            Pool p;
            const int64_t ldx = c.H + c.pad, ldg = 2 * c.I + c.pad;
            const int64_t hb = ck::fp8_blocks(c.H), ib = c.I / 128;
            uint16_t *x = p.get<uint16_t>(((c.M - 1) * ldx + c.H) * 2), *out = p.get<uint16_t>(((c.M - 1) * ldx + c.H) * 2);
            uint8_t *w1 = p.get<uint8_t>(2 * c.I * c.H), *s1 = p.get<uint8_t>(2 * ib * hb);
            uint8_t *w2 = p.get<uint8_t>(c.H * c.I), *s2 = p.get<uint8_t>(ib * hb);
            uint16_t *gu = p.get<uint16_t>(((c.M - 1) * ldg + 2 * c.I) * 2);
            const size_t need = ck_fp8_ffn_workspace_bytes(c.M, c.H, c.I);
            const size_t back = ck_fp8_ffn_backward_workspace_bytes(c.M, c.H, c.I);
            uint8_t *ws = p.get<uint8_t>((int64_t)need), *wb = p.get<uint8_t>((int64_t)back);
            EXPECT(need > 0 && need % 256 == 0 && back >= need && back % 256 == 0);
            const auto forward = [&](size_t bytes) {
                return ck_fp8_ffn(x, c.M, c.H, ldx, c.I, w1, s1, w2, s2, out, ldx, keep ? gu : nullptr, ldg, ws, bytes,
                                  nullptr);
            };
            const auto backward = [&](size_t bytes) {
                return ck_fp8_ffn_backward(x, c.M, c.H, ldx, gu, ldg, c.I, w1, s1, w2, s2, out, ldx, wb, bytes, nullptr);
            };
            runs([&] { return forward(need); });
            runs([&] { return backward(back); });
            g_calls = 0;
            EXPECT(forward(need - 1) == CK_ERR_WORKSPACE && backward(back - 1) == CK_ERR_WORKSPACE && g_calls == 0);
        }
}

// Every size gets a tile that its kind has, in a grid that one launch takes.
void tiles()
{
    const struct {
        ck::Fp8Tile tile;
        int64_t n, m;
    } sizes[] = {{ck::Fp8Tile::k256x256, 256, 256}, {ck::Fp8Tile::k256x192, 256, 192}, {ck::Fp8Tile::k256x128, 256, 128},
                 {ck::Fp8Tile::k256x64, 256, 64},   {ck::Fp8Tile::k128x128, 128, 128}, {ck::Fp8Tile::k128x64, 128, 64},
                 {ck::Fp8Tile::k64x64, 64, 64}};
    bool seen[3][7] = {};
    for (int64_t M = 1; M < (int64_t(1) << 31); M = M * 5 / 4 + 1)
        for (int64_t N = 16; N < (int64_t(1) << 31); N = N * 3 / 2 / 16 * 16 + 16)
            for (int kind = 0; kind < 3; ++kind) {
                const int64_t columns = kind == 0 ? N : (N + 127) / 128 * 128;
                if (ck::fp8_tiles(M, columns * (kind == 1 ? 2 : 1)) > ck::kFp8MaxTiles)
                    continue;
                const ck::Fp8Plan plan = ck::fp8_plan((ck::Fp8Result)kind, M, 2048, columns, false);
                EXPECT(plan.splits == 1 && plan.each == 16);
                bool found = false;
                for (int i = 0; i < 7; ++i)
                    if (sizes[i].tile == plan.tile) {
                        found = seen[kind][i] = true;
                        const int64_t rows = columns * (kind == 1 ? 2 : 1);
                        const int64_t grid = (rows + sizes[i].n - 1) / sizes[i].n * ((M + sizes[i].m - 1) / sizes[i].m);
                        EXPECT(plan.time > 0 && grid * 512 < (int64_t(1) << 32));
                        EXPECT(kind != 1 || sizes[i].n == 256);   // whole blocks of gate and up
                        EXPECT(kind != 2 || sizes[i].n >= 128);
                    }
                EXPECT(found);
            }
    EXPECT(ck::fp8_split_floats(INT32_MAX, 32768, INT32_MAX) == ck::kFp8SplitArea);
    EXPECT(ck::fp8_split_floats(1, 32768, INT32_MAX) == ck::kFp8SplitArea && ck::fp8_split_floats(1, 1024, 4096) == 0);
    // Room for a smaller call's sums is in a larger call's.
    for (int64_t K = 16; K <= 32768; K += 2032)
        for (int64_t N = 16; N < 40000; N = N * 3 / 16 * 8 + 16) {
            int64_t room = 0;
            for (int64_t M = 1; M < 5000; ++M) {
                EXPECT(ck::fp8_split_floats(M, K, N) >= room);
                room = ck::fp8_split_floats(M, K, N);
                const ck::Fp8Plan plan = ck::fp8_plan(ck::Fp8Result::kBf16, M, K, N, true);
                const int64_t n = plan.tile == ck::Fp8Tile::k64x64 ? 64 : 128, m = plan.tile == ck::Fp8Tile::k128x128 ? 128 : 64;
                EXPECT(plan.splits == 1 || plan.splits * ((N + n - 1) / n * n) * ((M + m - 1) / m * m) <= room);
            }
        }
    for (int kind = 0; kind < 3; ++kind)
        for (int i = 0; i < 7; ++i)
            EXPECT(seen[kind][i] == (kind == 1 ? sizes[i].n == 256 : i != 3 && (kind == 0 || i != 6)));
}

}  // namespace

int main()
{
    linears();
    blocks();
    tiles();
    printf("fp8 driver: %d checks, %d failures\n", g_checks, g_failures);
    return g_failures ? 1 : 0;
}
