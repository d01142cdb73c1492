// Internal launch interface of the 8-bit float operators (quantisers, products with a
// scale for each block of 128, the gated feed-forward block), between ck_fp8_api.cpp
// and their kernels.  Arguments were validated by the caller; each launcher returns
// the hipError_t of its launches as an int (0 = success).
//
// Codes are e4m3 bytes, scales e8m0 bytes (2^(byte - 127)).  Activations: codes
// [M, lda], scales [M, ldsa], one for each 128 columns, rows 4-byte aligned and ldsa % 4
// == 0.  Weights: codes [N, ldw], scales dense [ceil(N / 128), ceil(K / 128)].
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ck {

constexpr int kFp8Block = 128;
inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }
// Row stride in bytes of an activation's scales in a workspace.
inline int64_t fp8_scale_stride(int64_t K) { return (fp8_blocks(K) + 3) / 4 * 4; }

int launch_fp8_quant(const void *x, bool f32, int64_t M, int K, int64_t ldx, uint8_t *codes, int64_t lda,
                     uint8_t *scales, int64_t ldsa, void *stream);
int launch_fp8_quantize_weights(const uint16_t *w, int64_t N, int K, int64_t ldw_in, uint8_t *codes, int64_t ldw,
                                uint8_t *scales, void *stream);
int launch_fp8_transpose(const uint8_t *codes, int64_t ldw, const uint8_t *scales, int N, int K, uint8_t *codes_t,
                         int64_t ldt, uint8_t *scales_t, void *stream);

// What a product's sums become.
enum class Fp8Result {
    kBf16,   // bf16 (sums + bias)
    kGated,  // of 2 I weight rows, gate then up: silu(g) u, quantised; g and u in bf16 where gate_up is given
    kGrad,   // d(gate) and d(up) of silu(g) u from sums dh and given g and u, quantised
};
struct Fp8Product {
    const uint8_t *a, *sa;   // activations
    int64_t lda, ldsa;
    int64_t M;
    int K;
    const uint8_t *w, *sw;   // weights
    int64_t ldw;
    int N;                   // weight rows
    // kBf16
    const uint16_t *bias;
    uint16_t *out;
    int64_t ldo;
    // kGated, kGrad: I columns of h, or of dg and of du
    int I;
    uint16_t *gate_up;       // bf16 [M, ldg]: g at column 0, u at column I
    int64_t ldg;
    uint8_t *q, *sq;         // the quantised result [M, I] or [M, 2 I]
    int64_t ldsq;
};
// Tiles of the tiled product, weight rows x activation rows: 256 x 256, 256 x 128, 128 x 128
// (two workgroups a CU; not for kGated, whose tiles cover 128 columns of gate and of up).
enum class Fp8Tile { k256x256, k256x192, k256x128, k256x64, k128x128, k128x64, k64x64 };
constexpr int kFp8Cus = 256;
// Workgroups of 512 threads that one launch takes, and those of a product on 128 x 128 tiles, which
// the entry points hold against it.
constexpr int64_t kFp8MaxTiles = (int64_t(1) << 32) / 512 - 1;
inline int64_t fp8_tiles(int64_t M, int64_t N) { return fp8_blocks(M) * fp8_blocks(N); }
// The tile with the least rounds times time of a step: those of the table, in hundredths of a
// microsecond, with a workgroup on every CU.  Measured, the quantiser included, in the table's
// order (256 x 64 only for kGated, which has none below): 128 x 3840 x 10240 (rows, K, N)
// 39.0 / 34.0 / 26.3 / - / 18.9 / 16.0 / 18.5 us, 256 x 3840 x 3840 39.6 / 34.6 / 26.5 / - / 19.0 /
// 16.0 / 14.3, 512 x 10240 x 3840 91.0 / 77.6 / 59.3 / - / 40.9 / 36.4 / 42.2, 700 x 3840 x 3840
// 40.6 / 35.3 / 27.6 / - / 21.7 / 28.2 / 27.6, 2048 x 3840 x 3840 45.7 / 41.5 / 36.8 / - / 43.2 /
// 56.2 / 60.3, 2000 x 3840 x 10240 92 / 83 / 92 / - / 99 / 131 / 140, 8192 x 10240 x 3840 286 / 326 /
// 346 / - / 416 / 528 / 576.  Feed-forward block of 77 rows, H 2112, I 1280: 31.4 / 28.7 / 23.5 /
// 20.1; of 2000, H 2048, I 5120: 81.6 / 78.1 / 81.8 / 90.9.
struct Fp8Plan {
    Fp8Tile tile;
    int64_t cost;   // of a step
};
inline Fp8Plan fp8_plan(Fp8Result kind, int64_t M, int64_t columns)
{
    struct Shape {
        Fp8Tile tile;
        int n, m, cost;
    };
    constexpr Shape shapes[] = {
        {Fp8Tile::k256x256, 256, 256, 140}, {Fp8Tile::k256x192, 256, 192, 120}, {Fp8Tile::k256x128, 256, 128, 100},
        {Fp8Tile::k256x64, 256, 64, 70},    {Fp8Tile::k128x128, 128, 128, 60},  {Fp8Tile::k128x64, 128, 64, 46},
        {Fp8Tile::k64x64, 64, 64, 33},
    };
    const bool gated = kind == Fp8Result::kGated;
    Fp8Plan best{Fp8Tile::k256x256, INT64_MAX};
    for (const Shape &s : shapes) {
        if (gated ? s.n < 256 : s.n == 256 && s.m == 64)
            continue;
        if (kind == Fp8Result::kGrad && s.n < 128)
            continue;
        const int64_t tiles = (columns * (gated ? 2 : 1) + s.n - 1) / s.n * ((M + s.m - 1) / s.m);
        const int64_t cost = s.cost * ((tiles + kFp8Cus - 1) / kFp8Cus);
        if (cost < best.cost && tiles <= kFp8MaxTiles)
            best = Fp8Plan{s.tile, cost};
    }
    return best;
}
int launch_fp8_tiled(Fp8Result kind, const Fp8Product &p, void *stream);

// The few-row product.  x given: bf16 or fp32 rows, quantised on the way (fp8_few_raw), a and sa
// unused; null: the codes and scales.  kGated and kGrad write fp32 [M, I] or [M, 2 I] to sums.
constexpr int64_t kFp8FewRows = 64;
constexpr int kFp8RawRows = 8, kFp8RawBytes = 16 * 1024;
inline bool fp8_few_raw(int64_t M, int64_t K) { return M <= kFp8RawRows && M * (fp8_blocks(K) * 128) <= kFp8RawBytes; }
// Columns that rows of codes, in tiles of 16, take at most: wider ones the tiles do faster.
constexpr int64_t fp8_few_columns(Fp8Result kind, int64_t rows16)
{
    return kFp8Cus * 16 * (kind == Fp8Result::kGated || (kind == Fp8Result::kBf16 && rows16 > 2) ? 2 : 3);
}
// Whether it serves rows of codes: where the rows' scales fit LDS beside 128 KB of rings, and where it takes
// less time than the tiles, whose time is that of a step after a step.  Nanoseconds, lines through
// times that were measured; few rows / tiles in microseconds, both with the quantiser, (rows, K,
// N): 16 x 3840 x 3840 9.6 / 13.1, 64 x 3840 x 3840 13.0 / 13.3, 16 x 3840 x 10240 13.7 / 13.5,
// 48 x 10240 x 3840 17.2 / 25.5, 16 x 2112 x 1040 8.1 / 9.7, 32 x 2048 x 20480 18.9 / 12.7.
inline bool fp8_few(Fp8Result kind, int64_t M, int64_t K, int64_t columns)
{
    const int64_t rows16 = (M + 15) / 16;
    if (M > kFp8FewRows || M * fp8_scale_stride(K) > 16 * 1024 || columns > fp8_few_columns(kind, rows16))
        return false;
    const int64_t weights = K * columns * (kind == Fp8Result::kGated ? 2 : 1) / 1000;
    const int64_t quantiser = kind == Fp8Result::kBf16 ? 0 : 2500;   // of its fp32 results
    const int64_t few = 3600 + 600 * rows16 + weights * (140 + 28 * rows16) / 1000 + quantiser;
    return few < 3200 + 7 * fp8_blocks(K) * fp8_plan(kind, M, columns).cost;
}
int launch_fp8_few(Fp8Result kind, const Fp8Product &p, const void *x, bool f32, int64_t ldx, float *sums,
                   void *stream);

}  // namespace ck
