// Which forms of the 8-bit float product kernels calls of ck_fp8_api.cpp come to: the entry points
// run against stand-ins of their launchers, which touch no memory and print what they are asked for.
//   linear M K N | ffn M H I | backward M H I   (from standard input)   a line with the call's forms
//   sweep                                        every form that some size comes to, with one such call
// A few-row form is its source, result, 16-row tiles of activations and of weights a pass; a tiled form
// its tile and result, "sums" where K is split.  "passes": several; "runs": more than one run of scales.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <map>
#include <set>
#include <string>

#include "../../include/ck.h"
#include "../../packed_int4_convrot_amd/csrc/fp8_launch.h"

namespace {

std::set<std::string> g_forms;
const char *const kKinds[] = {"bf16", "gated", "grad", "sums"};

}  // namespace

namespace ck {

int launch_fp8_quant(const void *, bool, int64_t, int, int64_t, uint8_t *, int64_t, uint8_t *, int64_t, void *) { return 0; }
int launch_fp8_quantize_weights(const uint16_t *, int64_t, int, int64_t, uint8_t *, int64_t, uint8_t *, void *) { return 0; }
int launch_fp8_transpose(const uint8_t *, int64_t, const uint8_t *, int, int, uint8_t *, int64_t, uint8_t *, void *)
{
    return 0;
}

int launch_fp8_tiled(Fp8Result kind, const Fp8Product &p, const Fp8Plan &plan, float *, void *)
{
    static const char *const tiles[] = {"256x256", "256x192", "256x128", "256x64", "128x128", "128x64", "64x64"};
    const bool split = plan.splits > 1;
    g_forms.insert(std::string("tiled ") + tiles[(int)plan.tile] + " " + kKinds[split ? 3 : (int)kind] +
                   ((split ? plan.each : fp8_blocks(p.K)) > 64 ? " runs" : ""));
    return 0;
}

int launch_fp8_few(Fp8Result kind, const Fp8Product &p, const void *x, bool f32, int64_t, float *, void *)
{
    const int64_t rows16 = (p.M + 15) / 16;
    const Fp8FewRun run = fp8_few_run(x != nullptr, kind, rows16, kind == Fp8Result::kBf16 ? p.N : p.I);
    char form[64];
    snprintf(form, sizeof form, "few %s %s %d %d%s", x ? f32 ? "fp32" : "raw" : "codes", kKinds[(int)kind], (int)rows16,
             run.tiles, run.passes > 1 ? " passes" : "");
    g_forms.insert(form);
    return 0;
}

}  // namespace ck

namespace {

// Addresses that nothing reads, far enough apart for the largest call.
template <class T>
T *at(int i) { return reinterpret_cast<T *>((uintptr_t)(i + 1) << 42); }

constexpr size_t kRoom = (size_t)1 << 41;

// M, K, N or M, H, I.
int call(const std::string &op, int64_t M, int64_t K, int64_t N)
{
    g_forms.clear();
    if (op == "linear") {
        const int64_t lds = ck::fp8_scale_stride(K);
        const int e = ck_fp8_gemm(at<uint8_t>(0), K, at<uint8_t>(1), lds, M, K, at<uint8_t>(2), K, at<uint8_t>(3), N, nullptr,
                                  at<uint16_t>(4), N, nullptr);
        return e ? e : ck_fp8_linear(at<uint16_t>(0), M, K, K, at<uint8_t>(2), K, at<uint8_t>(3), N, nullptr, at<uint16_t>(4),
                                     N, at<void>(5), kRoom, nullptr);
    }
    if (op == "ffn")
        return ck_fp8_ffn(at<uint16_t>(0), M, K, K, N, at<uint8_t>(1), at<uint8_t>(2), at<uint8_t>(3), at<uint8_t>(4),
                          at<uint16_t>(5), K, nullptr, 0, at<void>(6), kRoom, nullptr);
    return ck_fp8_ffn_backward(at<uint16_t>(0), M, K, K, at<uint16_t>(7), 2 * N, N, at<uint8_t>(1), at<uint8_t>(2),
                               at<uint8_t>(3), at<uint8_t>(4), at<uint16_t>(5), K, at<void>(6), kRoom, nullptr);
}

// Multiples of `of` from `lo` to `hi`, a step of 1 / `part` or so apart.
std::set<int64_t> spread(int64_t lo, int64_t hi, int64_t of, int64_t part)
{
    std::set<int64_t> s{hi};
    for (int64_t v = lo; v < hi; v += (v / part + of) / of * of)
        s.insert(v);
    return s;
}

void sweep()
{
    std::map<std::string, std::string> seen;
    std::set<int64_t> rows = spread(70, 20000, 1, 7);
    for (int64_t M = 1; M < 70; ++M)
        rows.insert(M);
    std::set<int64_t> K = spread(16, 32768, 16, 4);
    for (int64_t k : {8192, 8208, 16384, 16400})
        K.insert(k);
    const std::set<int64_t> N = spread(16, 140000, 16, 5), I = spread(128, 32768, 128, 6);
    for (const char *op : {"linear", "ffn", "backward"})
        for (int64_t M : rows)
            for (int64_t k : K)
                for (int64_t n : strcmp(op, "linear") == 0 ? N : I) {
                    if (call(op, M, k, n) != 0) {
                        fprintf(stderr, "refused: %s %lld %lld %lld: %s\n", op, (long long)M, (long long)k, (long long)n,
                                ck_last_error_msg());
                        continue;
                    }
                    for (const std::string &f : g_forms)
                        if (!seen.count(f))
                            seen[f] = std::string(op) + " " + std::to_string(M) + " " + std::to_string(k) + " " +
                                      std::to_string(n);
                }
    for (const auto &f : seen)
        printf("%s: %s\n", f.first.c_str(), f.second.c_str());
}

}  // namespace

int main()
{
    char op[32];
    long long M, K, N;
    while (scanf("%31s", op) == 1) {
        if (strcmp(op, "sweep") == 0) {
            sweep();
            continue;
        }
        if (scanf("%lld %lld %lld", &M, &K, &N) != 3 || call(op, M, K, N) != 0) {
            printf("refused: %s\n", ck_last_error_msg());
            continue;
        }
        for (const std::string &f : g_forms)
            printf("%s; ", f.c_str());
        printf("\n");
    }
    return 0;
}
