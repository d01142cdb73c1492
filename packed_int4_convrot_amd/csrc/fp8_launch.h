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
enum class Fp8Tile { kLarge, kMiddle, kSmall };
constexpr int kFp8Cus = 256;
// Workgroups of the product on the smallest tiles.
inline int64_t fp8_tiles(int64_t M, int64_t N) { return fp8_blocks(M) * fp8_blocks(N); }
// The tile with the least rounds times time of a step's tile on a full chip (hundredths of a
// microsecond: 140, 100, and 106 for two small ones or 55 for one a CU).  Measured, the
// quantiser included, large / middle / small: 512 x 3840 x 3840 (rows, K, N) 40 / 27 / 21 us,
// 512 x 3840 x 10240 41 / 30 / 32, 1024 x 3840 x 10240 45 / 54 / 50, 2048 x 10240 x 3840
// 99 / 84 / 90, 4096 x 3840 x 3840 59 / 69 / 72, 8192 x 3840 x 3840 118 / 137 / 141.
inline Fp8Tile fp8_tile(Fp8Result kind, int64_t M, int64_t columns)
{
    const int64_t wide = (columns * (kind == Fp8Result::kGated ? 2 : 1) + 255) / 256;
    const int64_t large = wide * ((M + 255) / 256), middle = wide * fp8_blocks(M);
    const int64_t small = kind == Fp8Result::kGated ? INT32_MAX : fp8_tiles(M, columns);
    auto rounds = [](int64_t tiles, int64_t slots) { return (tiles + slots - 1) / slots; };
    const int64_t cost_large = 140 * rounds(large, kFp8Cus), cost_middle = 100 * rounds(middle, kFp8Cus);
    const int64_t cost_small = small <= kFp8Cus ? 55 : 106 * rounds(small, 2 * kFp8Cus);
    if (cost_small < cost_middle && cost_small < cost_large)
        return Fp8Tile::kSmall;
    return cost_middle < cost_large ? Fp8Tile::kMiddle : Fp8Tile::kLarge;
}
int launch_fp8_tiled(Fp8Result kind, const Fp8Product &p, void *stream);

// Rows up to which the few-row product serves (64 x 3840 x 10240: 18.7 us against 19.5 of small
// tiles; 100 x 3840 x 3840 19.9 against 19.5, 128 x 3840 x 10240 30.7 against 20.0).
// x given: bf16 or fp32 rows, quantised on the way (fp8_few_raw), a and sa unused;
// null: the codes and scales.  kGated and kGrad write fp32 [M, I] or [M, 2 I] to sums.
constexpr int64_t kFp8FewRows = 64;
constexpr int kFp8RawRows = 8, kFp8RawBytes = 16 * 1024;
inline bool fp8_few_raw(int64_t M, int64_t K) { return M <= kFp8RawRows && M * (fp8_blocks(K) * 128) <= kFp8RawBytes; }
// The rows' scales lie in LDS beside 128 KB of rings.
inline bool fp8_few(int64_t M, int64_t K) { return M <= kFp8FewRows && M * fp8_scale_stride(K) <= 16 * 1024; }
int launch_fp8_few(Fp8Result kind, const Fp8Product &p, const void *x, bool f32, int64_t ldx, float *sums,
                   void *stream);

}  // namespace ck
