// Drives the entry points of ck_rows_api.cpp against host stand-ins for their
// launchers, under AddressSanitizer and UndefinedBehaviorSanitizer.  The
// stand-ins touch the first and the last byte of everything the kernels may
// reach, in buffers of exactly the documented sizes, and check what a launcher
// may rely on: at most kMoePairs pairs a pass, room for them in the workspace,
// every token in one pass.
// Prints "rows driver: N checks, 0 failures" and exits 0 when all pass.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <initializer_list>
#include <vector>

#include "../../include/ck.h"
#include "../../packed_int4_convrot_amd/csrc/rows_launch.h"

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

int g_calls, g_next_status;
int64_t g_tokens;
const void *g_expected_x;  // of the next pass

}  // namespace

namespace ck {

int launch_moe_route(const void *logits, bool bf16, int64_t T, int E, int64_t ldl, int k, bool, int32_t *ids,
                     float *weights, void *)
{
    ++g_calls;
    read_span(logits, T, E, ldl, bf16 ? 2 : 4);
    write_span(ids, T, k, k, 4);
    write_span(weights, T, k, k, 4);
    const int e = g_next_status;
    g_next_status = 0;
    return e;
}

int launch_moe(const uint16_t *x, int T, int64_t ldx, const MoeRouting &r, const MoeExperts &w, uint16_t *out,
               int64_t ldo, void *ws, void *)
{
    ++g_calls;
    const int64_t P = (int64_t)T * r.k;
    EXPECT(T >= 1 && P <= kMoePairs);
    EXPECT(x == g_expected_x);
    g_expected_x = x + T * ldx;
    g_tokens += T;
    read_span(x, T, w.H, ldx, 2);
    if (r.logits) {
        read_span(r.logits, T, w.E, r.ldl, r.bf16 ? 2 : 4);
        write_span(r.ids, T, r.k, r.k, 4);
        write_span(r.weights, T, r.k, r.k, 4);
    } else {
        read_span(r.ids, T, r.k, r.k, 4);
        read_span(r.weights, T, r.k, r.k, 4);
    }
    read_span(w.w1, (int64_t)w.E * 2 * w.I, w.H / 2, w.H / 2, 1);
    read_span(w.s1, (int64_t)w.E * (w.H / 64), 2 * w.I, 2 * w.I, 2);
    read_span(w.z1, (int64_t)w.E * (w.H / 64), 2 * w.I, 2 * w.I, 2);
    read_span(w.w2, (int64_t)w.E * w.H, w.I / 2, w.I / 2, 1);
    read_span(w.s2, (int64_t)w.E * (w.I / 64), w.H, w.H, 2);
    read_span(w.z2, (int64_t)w.E * (w.I / 64), w.H, w.H, 2);
    write_span(ws, 1, moe_hidden_bytes(P, w.I), 0, 1);
    write_span(static_cast<uint8_t *>(ws) + moe_hidden_bytes(P, w.I), P, w.H, w.H, 4);
    write_span(out, T, w.H, ldo, 2);
    const int e = g_next_status;
    g_next_status = 0;
    return e;
}

int launch_lora(const uint16_t *x, int64_t M, int K, int64_t ldx, const int32_t *index, int64_t L, int R,
                const uint16_t *a, const uint16_t *b, const float *scaling, const int32_t *ranks, int N,
                const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo, float *ws, void *)
{
    ++g_calls;
    read_span(x, M, K, ldx, 2);
    read_span(index, 1, M, M, 4);
    read_span(a, L * R, K, K, 2);
    read_span(b, L * N, R, R, 2);
    read_span(scaling, 1, L, L, 4);
    read_span(ranks, 1, L, L, 4);
    read_span(base, M, N, ldb, 2);
    write_span(ws, (int64_t)lora_splits(M, K, R, L) * M, R, R, 4);
    write_span(out, M, N, ldo, 2);
    const int e = g_next_status;
    g_next_status = 0;
    return e;
}

}  // namespace ck

namespace {

void routes()
{
    for (int kind : {CK_LOGITS_F32, CK_LOGITS_BF16})
        for (int64_t T : {1, 5, 700})
            for (int64_t E : {1, 60, 1024})
                for (int k : {1, 8, 32})
                    for (int64_t pad : {0, 3}) {
                        Pool p;
                        const int64_t size = kind == CK_LOGITS_BF16 ? 2 : 4;
                        void *l = p.get<uint8_t>(((T - 1) * (E + pad) + E) * size);
                        memset(l, 0, (size_t)(((T - 1) * (E + pad) + E) * size));
                        int32_t *ids = p.get<int32_t>(T * k * 4);
                        float *w = p.get<float>(T * k * 4);
                        g_calls = 0;
                        EXPECT(ck_moe_route(l, kind, T, E, E + pad, k, 1, ids, w, nullptr) == CK_OK && g_calls == 1);
                        g_next_status = 1;
                        EXPECT(ck_moe_route(l, kind, T, E, E + pad, k, 0, ids, w, nullptr) == CK_ERR_HIP);
                        EXPECT(ck_last_error_msg()[0] != 0);
                        EXPECT(ck_moe_route(l, kind, T, E, E - 1, k, 0, ids, w, nullptr) == CK_ERR_INVALID_ARG);
                        EXPECT(ck_moe_route(l, kind, T, E, E + pad, k, 0, ids, (float *)ids, nullptr) ==
                               CK_ERR_INVALID_ARG);
                        EXPECT(g_calls == 2);
                    }
}

void layers()
{
    const struct {
        int64_t T, H, I, E;
        int k;
        int64_t pad;
        bool zeros;
    } cases[] = {{1, 64, 64, 1, 1, 0, true},      {3, 256, 128, 8, 2, 8, false},  {37, 128, 192, 5, 8, 0, true},
                 {128, 64, 64, 3, 8, 0, true},    {129, 64, 64, 3, 8, 16, true},  {300, 64, 128, 4, 7, 0, false},
                 {33, 64, 64, 40, 32, 0, true},   {2, 32768, 64, 2, 32, 0, true}, {9, 32768, 64, 2, 1, 8, true},
                 {2, 64, 32768, 1, 3, 0, false},  {1100, 64, 64, 2, 1, 0, true},  {40, 16384, 64, 2, 30, 0, true}};
    for (const auto &c : cases) {
        Pool p;
        const int64_t ldx = c.H + c.pad, ldl = c.E + c.pad;
        uint16_t *x = p.get<uint16_t>(((c.T - 1) * ldx + c.H) * 2), *out = p.get<uint16_t>(((c.T - 1) * ldx + c.H) * 2);
        float *l = p.get<float>(((c.T - 1) * ldl + c.E) * 4), *w = p.get<float>(c.T * c.k * 4);
        int32_t *ids = p.get<int32_t>(c.T * c.k * 4);
        uint8_t *w1 = p.get<uint8_t>(c.E * c.I * c.H), *w2 = p.get<uint8_t>(c.E * c.H * c.I / 2);
        const int64_t n1 = c.E * (c.H / 64) * 2 * c.I * 2, n2 = c.E * (c.I / 64) * c.H * 2;
        uint16_t *s1 = p.get<uint16_t>(n1), *s2 = p.get<uint16_t>(n2);
        uint16_t *z1 = c.zeros ? p.get<uint16_t>(n1) : nullptr, *z2 = c.zeros ? p.get<uint16_t>(n2) : nullptr;
        const size_t need = ck_moe_workspace_bytes(c.T, c.I, c.E, c.k);
        uint8_t *ws = p.get<uint8_t>((int64_t)need);
        EXPECT(need > 0 && need % 256 == 0);
        const auto layer = [&](size_t bytes) {
            g_calls = 0, g_tokens = 0, g_expected_x = x;
            return ck_moe_w4a16(x, c.T, c.H, ldx, l, CK_LOGITS_F32, ldl, c.k, 1, c.E, c.I, 64, w1, s1, z1, w2, s2, z2,
                                out, ldx, ids, w, ws, bytes, nullptr);
        };
        EXPECT(layer(need) == CK_OK && g_tokens == c.T);
        const int passes = g_calls;
        EXPECT(layer(need - 1) == CK_ERR_WORKSPACE && g_calls == 0);
        g_next_status = 7;
        EXPECT(layer(need) == CK_ERR_HIP && g_calls == 1);
        g_calls = 0, g_tokens = 0, g_expected_x = x;
        EXPECT(ck_moe_experts_w4a16(x, c.T, c.H, ldx, ids, w, c.k, c.E, c.I, 64, w1, s1, z1, w2, s2, z2, out, ldx, ws,
                                    need, nullptr) == CK_OK);
        EXPECT(g_tokens == c.T && g_calls == passes);
    }
}

void adapters()
{
    const struct {
        int64_t M, K, R, L, N, pad;
    } cases[] = {{1, 64, 8, 1, 16, 0},      {1, 3840, 16, 3, 512, 0}, {17, 192, 24, 2, 272, 8}, {64, 128, 64, 5, 128, 0},
                 {65, 448, 72, 9, 160, 16}, {1024, 64, 256, 2, 16, 0}, {1025, 192, 24, 3, 528, 8}, {3000, 64, 64, 300, 16, 0}};
    for (const auto &c : cases)
        for (bool optional : {true, false}) {
            Pool p;
            const int64_t ldx = c.K + c.pad, ldo = c.N + c.pad, ldb = c.N + 2 * c.pad;
            uint16_t *x = p.get<uint16_t>(((c.M - 1) * ldx + c.K) * 2);
            uint16_t *out = p.get<uint16_t>(((c.M - 1) * ldo + c.N) * 2);
            uint16_t *base = optional ? p.get<uint16_t>(((c.M - 1) * ldb + c.N) * 2) : nullptr;
            uint16_t *a = p.get<uint16_t>(c.L * c.R * c.K * 2), *b = p.get<uint16_t>(c.L * c.N * c.R * 2);
            float *scaling = optional ? p.get<float>(c.L * 4) : nullptr;
            int32_t *ranks = optional ? p.get<int32_t>(c.L * 4) : nullptr, *index = p.get<int32_t>(c.M * 4);
            const size_t need = ck_lora_workspace_bytes(c.M, c.K, c.R, c.L);
            uint8_t *ws = p.get<uint8_t>((int64_t)need);
            const auto add = [&](const uint16_t *y, int64_t ldy, size_t bytes) {
                g_calls = 0;
                return ck_lora_add(x, c.M, c.K, ldx, index, c.L, c.R, a, b, scaling, ranks, c.N, y, ldy, out, ldo, ws,
                                   bytes, nullptr);
            };
            EXPECT(add(base, ldb, need) == CK_OK && g_calls == 1);
            EXPECT(add(out, ldo, need) == CK_OK && g_calls == 1);
            EXPECT(add(out, ldo + 8, need) == CK_ERR_INVALID_ARG && g_calls == 0);
            EXPECT(add(base, ldb, need - 1) == CK_ERR_WORKSPACE && g_calls == 0);
            g_next_status = 7;
            EXPECT(add(base, ldb, need) == CK_ERR_HIP && g_calls == 1);
        }
}

}  // namespace

int main()
{
    routes();
    layers();
    adapters();
    printf("rows driver: %d checks, %d failures\n", g_checks, g_failures);
    return g_failures ? 1 : 0;
}
