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
    kSums,   // fp32, a tile's as the matrix core leaves them: part of a split kBf16
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
    // kSums: steps of a split, and the splits' sums
    int each;
    float *sums;
};
// Tiles of the tiled product, weight rows x activation rows.  kGated's cover 128 columns of gate and of
// up, so it has those of 256 weight rows, 256 x 64 by itself; kGrad has no 64 x 64, half a block of 128.
enum class Fp8Tile { k256x256, k256x192, k256x128, k256x64, k128x128, k128x64, k64x64 };
constexpr int kFp8Cus = 256;
// Workgroups of 512 threads that one launch takes, and those of a product on 128 x 128 tiles, which
// the entry points hold against it.
constexpr int64_t kFp8MaxTiles = (int64_t(1) << 32) / 512 - 1;
inline int64_t fp8_tiles(int64_t M, int64_t N) { return fp8_blocks(M) * fp8_blocks(N); }
// The plan that takes the least time: 3200 ns (1000 more with the activation), and for each round
// of tiles over the CUs and each step of 128 columns 7 ns times the cost in the table below.
// Measured in us, the quantiser included, on 256 x 256 / 256 x 192 / 256 x 128 / 128 x 128 / 128 x 64 /
// 64 x 64 tiles, whole (rows x K x N):
//    128 x  3840 x 10240   39.0 / 34.0 / 26.3 / 18.9 / 16.0 / 18.5
//    256 x  3840 x  3840   39.6 / 34.6 / 26.5 / 19.0 / 16.0 / 14.3
//    700 x  3840 x  3840   40.6 / 35.3 / 27.6 / 21.7 / 28.2 / 27.6
//   2048 x  3840 x  3840   45.7 / 41.5 / 36.8 / 43.2 / 56.2 / 60.3
//   2000 x  3840 x 10240   92 / 83 / 92 / 99 / 131 / 140
//   8192 x 10240 x  3840   286 / 326 / 346 / 416 / 528 / 576
// and with 256 x 256 / 256 x 192 / 256 x 128 / 256 x 64 under the activation, feed-forward blocks (rows,
// H, I): 77, 2112, 1280 31.4 / 28.7 / 23.5 / 20.1; 2000, 2048, 5120 81.6 / 78.1 / 81.8 / 90.9.
//
// kBf16 on the three smallest tiles may split K over `splits` workgroups, each of `each` steps (a
// multiple of four), whose fp32 sums go through the workspace and a launch that adds them: 1900 ns,
// and 2.5 for a thousand sums.  Whole / split: 100 x 10240 x 3840 26.4 / 18.2, 100 x 20480 x 3840
// 47.2 / 25.7, 128 x 8192 x 1024 22.9 / 13.1, 2000 x 20480 x 256 64 / 43, 100 x 3840 x 1040 13.2 / 11.2,
// 200 x 20480 x 3840 49.5 / 37.3 on 128 x 64, 34.8 on 128 x 128;
// 100 x 2112 x 1040 stays whole, 10.0 / 10.6.  Backward pass of 100 rows, H 3840, I 10240: 68.6 / 49.4.
//
// The lines are of tiles on a part of the chip, weights in a cache.  With nearly all CUs at work they
// fall short of the time: 300 x 3840 x 10240 15.8 us where the product takes 18.2 (20.5 with weights from
// memory), 1000 x 3840 x 3840 15.8 of 19.7 (21.6), 2000 x 5120 x 2048 20.0 of 25.1 (28.3), all on 128 x 128
// tiles.  The table's times, not these sums, say which tile is the faster one there.
struct Fp8Plan {
    Fp8Tile tile;
    int64_t splits, each;
    int64_t time;
};
constexpr int64_t kFp8MostSplits = 8, kFp8SplitArea = int64_t(kFp8Cus) * 128 * 128;   // elements of all sums
// Floats that a split product's sums need at most (up to 64 rows take no 128 x 128 tiles).  Fewer
// rows need no more.
inline int64_t fp8_split_floats(int64_t M, int64_t K, int64_t N)
{
    const int64_t m = M <= 64 ? 64 : M < (1 << 15) ? fp8_blocks(M) * 128 : 1 << 15;
    const int64_t n = N < (1 << 15) ? fp8_blocks(N) * 128 : 1 << 15;
    const int64_t most = kFp8MostSplits * m * n;
    return K < 16 * kFp8Block ? 0 : most < kFp8SplitArea ? most : kFp8SplitArea;
}
inline Fp8Plan fp8_plan(Fp8Result kind, int64_t M, int64_t K, int64_t columns, bool may_split)
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
    const int64_t steps = fp8_blocks(K);
    Fp8Plan best{Fp8Tile::k256x256, 1, steps, INT64_MAX};
    for (const Shape &s : shapes) {
        if (gated ? s.n < 256 : s.n == 256 && s.m == 64)
            continue;
        if (kind == Fp8Result::kGrad && s.n < 128)
            continue;
        const int64_t tiles = (columns * (gated ? 2 : 1) + s.n - 1) / s.n * ((M + s.m - 1) / s.m);
        if (tiles > kFp8MaxTiles)
            continue;
        const bool splits = may_split && kind == Fp8Result::kBf16 && s.n < 256 && K >= 16 * kFp8Block;
        for (int64_t n = 1; n <= (splits ? kFp8MostSplits : 1) && (n == 1 || n * tiles <= kFp8Cus); ++n) {
            const int64_t each = n == 1 ? steps : ((steps + n - 1) / n + 3) / 4 * 4;
            const int64_t rounds = (tiles + kFp8Cus - 1) / kFp8Cus;
            const int64_t join = n == 1 ? 0 : 1900 + n * tiles * s.m * s.n / 400;
            const int64_t time = (gated ? 4200 : 3200) + 7 * s.cost * each * rounds + join;
            if (time < best.time)
                best = Fp8Plan{s.tile, (steps + each - 1) / each, each, time};
        }
    }
    return best;
}
int launch_fp8_tiled(Fp8Result kind, const Fp8Product &p, const Fp8Plan &plan, float *sums, void *stream);

// The few-row product.  x given: bf16 rows, or fp32 ones for kBf16, quantised on the way (fp8_few_raw),
// a and sa unused; null: the codes and scales.  kGated and kGrad write fp32 [M, I] or [M, 2 I] to sums.
constexpr int64_t kFp8FewRows = 64;
constexpr int kFp8RawRows = 8, kFp8RawBytes = 16 * 1024;
inline bool fp8_few_raw(int64_t M, int64_t K) { return M <= kFp8RawRows && M * (fp8_blocks(K) * 128) <= kFp8RawBytes; }
// Columns that rows of codes, in tiles of 16, take at most: wider ones the tiles do faster.
constexpr int64_t fp8_few_columns(Fp8Result kind, int64_t rows16)
{
    const int most = rows16 == 1 ? 3 : rows16 == 2 ? 2 : 1;
    return kFp8Cus * 16 * (kind == Fp8Result::kBf16 ? most : most < 3 ? most + 1 : 3);
}
// Whether it serves rows of codes: where the rows' scales fit LDS beside 128 KB of rings, and where
// it takes less time than the tiles.  Both in nanoseconds, lines through measured times: the weights'
// way from memory, every workgroup's way through all rows, the quantiser of fp32 results.
// Measured in us, few rows / tiles, both with the quantiser (rows x K x N), weights in a cache:
// 16 x 3840 x 3840 9.0 / 11.9, 64 x 3840 x 3840 13.3 / 12.2, 16 x 3840 x 10240 13.4 / 13.6, 64 x 10240 x 3840
// 19.1 / 16.0; weights from memory: 16 x 3840 x 3840 10.4 / 12.8, 16 x 3840 x 10240 14.9 / 16.1, 64 x 10240 x
// 3840 23.7 / 20.0; feed-forward block of 16 rows, H 3840, I 10240: 40.8 / 48.2, of 64 rows 55.7 / 51.7.
inline bool fp8_few(Fp8Result kind, int64_t M, int64_t K, int64_t columns, const Fp8Plan &plan)
{
    const int64_t rows16 = (M + 15) / 16;
    if (M > kFp8FewRows || M * fp8_scale_stride(K) > 16 * 1024 || columns > fp8_few_columns(kind, rows16))
        return false;
    const int64_t weights = columns * (kind == Fp8Result::kGated ? 2 : 1), tiles = (weights + 4095) / 4096;
    const int64_t quantiser = kind == Fp8Result::kBf16 ? 0 : 1500;   // of its fp32 results
    const int64_t few = 3800 + K * weights / 4600 + rows16 * (300 + 24 * fp8_blocks(K)) * (tiles + 3) / 4 + quantiser;
    const int64_t from_memory = 3200 + K * weights / 3300;
    return few < (plan.time > from_memory ? plan.time : from_memory);
}
// 16-row tiles of weights (of gate, and as many of up) that one of its passes takes at most.  Codes take
// one pass: wider results are the tiled product's.
constexpr int fp8_few_most_tiles(bool raw, Fp8Result kind, int64_t rows16)
{
    return raw ? 8 / (kind == Fp8Result::kGated ? 2 : 1) : (int)(fp8_few_columns(kind, rows16) / kFp8Cus / 16);
}
// An equal run of columns for each workgroup, in equal passes; a kernel of 1, 2, 3, 4, 6 or 8 tiles a pass.
struct Fp8FewRun {
    int per, grid, passes, tiles;
};
inline Fp8FewRun fp8_few_run(bool raw, Fp8Result kind, int64_t rows16, int64_t columns)
{
    const int per = (int)((columns + kFp8Cus - 1) / kFp8Cus), grid = (int)((columns + per - 1) / per);
    const int tiles = (per + 15) / 16, most = fp8_few_most_tiles(raw, kind, rows16);
    const int passes = (tiles + most - 1) / most, each = (tiles + passes - 1) / passes;
    return {per, grid, passes, each + (each == 5 || each == 7)};
}
int launch_fp8_few(Fp8Result kind, const Fp8Product &p, const void *x, bool f32, int64_t ldx, float *sums,
                   void *stream);

}  // namespace ck
