// Internal launch interface of the operators that choose weights row by row
// (the mixture-of-experts layer and the low-rank adapters), between
// ck_rows_api.cpp and their kernels.  Arguments were validated by the caller;
// each launcher returns the hipError_t of its launches as an int (0 = success).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ck {

// ---- router -------------------------------------------------------------
constexpr int kRouteMaxExperts = 1024;  // 16 logits per lane of a wave
constexpr int kRouteMaxK = 32;
int launch_moe_route(const void *logits, bool bf16, int64_t T, int E, int64_t ldl, int k, bool renormalize,
                     int32_t *ids, float *weights, void *stream);

// ---- experts ------------------------------------------------------------
// One pass takes at most kMoePairs (token, slot) pairs, and at most 8192 result
// columns a pair on average; more tokens, or wider layers, run as several passes
// over the same workspace: the hidden activations of P pairs (two bf16 each),
// then their fp32 results.
constexpr int kMoePairs = 1024;
// Pairs up to which every pair streams its own expert's weights in two launches
// (H 3840, I 1280, 64 experts: 8 pairs 26 us, against 38 us for the four launches
// that share them; 16 pairs 48 against 53; 24 pairs 63 against 65, and repeated
// experts are read again for each).
constexpr int kMoeFewPairs = 16;
// Inner width up to which they do: the second of the two launches has a ring of three
// stages and the hidden activations of each of its eight waves in LDS (H 3840, 8 of 64
// experts, one token: I 1536 30 us, against 41 us for the four launches; I 1600 43 us).
constexpr int kMoeFewInner = 1536;
inline int64_t moe_hidden_bytes(int64_t P, int64_t I) { return (P * I * 4 + 255) / 256 * 256; }
inline int64_t moe_pass_columns(int64_t P) { return P * 8192; }

struct MoeExperts {
    const uint8_t *w1;          // [E, 2 I, H / 2]: I gate rows, then I up rows
    const uint16_t *s1, *z1;    // [E, H / 64, 2 I]; z1 may be null
    const uint8_t *w2;          // [E, H, I / 2]
    const uint16_t *s2, *z2;    // [E, I / 64, H]; z2 may be null
    int E, H, I;
};
// logits null: ids and weights are inputs; otherwise they are written.
struct MoeRouting {
    const void *logits;
    bool bf16, renormalize;
    int64_t ldl;
    int k;
    int32_t *ids;
    float *weights;
};
// One pass: T * k <= kMoePairs, T >= 1.
int launch_moe(const uint16_t *x, int T, int64_t ldx, const MoeRouting &r, const MoeExperts &w, uint16_t *out,
               int64_t ldo, void *ws, void *stream);

// ---- low-rank adapters --------------------------------------------------
constexpr int kLoraWindow = 64;     // rows that share one look at the adapter indices
constexpr int kLoraMaxRank = 256;
constexpr int kLoraRankBlock = 64;
// Rows up to which a workgroup is started for every tile a window can have (K = N =
// 3840, rank 64, 6 adapters in runs: 1024 rows 40 us, against 42 us of whole windows; 1500
// rows 47 against 43, 2048 54 against 46; rank 16 with N 10240 27 against 43, 37 against 44,
// 46 against 50).  Mixed rows would gain beyond, 90 against 120 us at 2048 rows of 8
// adapters, but batches that large are prompts, whose rows come in runs.
constexpr int64_t kLoraFewRows = 1024;
inline int64_t lora_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Tiles of 16 rows that the sets of a window can have, a set being the rows of one
// adapter (rows without one join the first): rows / 16 and 15 / 16 of a tile for each set.
inline int lora_slots(int64_t M, int64_t L)
{
    const int64_t rows = M < kLoraWindow ? M : kLoraWindow, sets = rows < L ? rows : L;
    return (int)((rows + 15 * sets) / 16);
}
constexpr int64_t kLoraCus = 256;
inline int64_t lora_most_splits(int64_t K) { return K / 256 < 1 ? 1 : K / 256 < 8 ? K / 256 : 8; }
// Parts the K columns are split into, so that few rows still fill the chip: about
// one workgroup for each of the 256 CUs; a wave keeps a 64-column group at least,
// and the second product adds at most 8 parts.  Of the tiles that a window's sets
// can have, rows of few adapters use some: six are counted.  Over 66 sizes (70 to 1000
// rows of 6 to 15 adapters, in runs and mixed, ranks 16 to 64) counting four or five
// takes 3 or 2 % less time on average, but up to 13 or 9 % more for mixed rows (400 rows
// of 10, K 10240: 34.4 and 33.0 us against 30.5); counting two as much on average and up
// to 26 % more, and ten 3 % more on average and up to 54 % (1000 rows of 15 in runs,
// K 10240: 83.6 against 54.4).
inline int lora_splits(int64_t M, int64_t K, int64_t R, int64_t L)
{
    const int64_t slots = M > kLoraFewRows ? 1 : lora_slots(M, L);
    const int64_t tiles = lora_ceil(M, kLoraWindow) * (M > kLoraWindow && L < 16 && slots > 6 ? 6 : slots);
    int64_t s = kLoraCus / (tiles * lora_ceil(R, kLoraRankBlock));
    const int64_t most = lora_most_splits(K);
    s = s > most ? most : s;
    return (int)(s < 1 ? 1 : s);
}
// Rows of v, over all parts, that the workspace has room for: lora_splits() * M at
// least, and no fewer for more rows or columns, so that a workspace of the largest
// call serves every smaller one.  (Several parts need parts * windows <= kLoraCus.)
inline int64_t lora_room_rows(int64_t M, int64_t K)
{
    const int64_t split = lora_most_splits(K) * M, most = kLoraCus * kLoraWindow;
    return M > most ? M : split < most ? split : most;
}
// Waves of a workgroup of the second product, up to kLoraFewRows rows.  A wave brings
// four rows of v to LDS at a time, so tiles of more rows take four waves, which share
// that work (K = N = 3840, one wave against four: 16 rows of one adapter of rank 16
// 14.0 against 9.3 us; 32 rows of 4 of rank 64 15.2 against 13.1; 301 of 7 22.7 against
// 18.7).  Tiles of one or two rows take one wave, whose workgroups spread over the chip
// (1 row of rank 16 8.0 against 8.4 us, of rank 64 10.8 against 12.2; 512 rows of 64
// adapters of rank 64 123 against 133), unless the chip is full anyway and the ranks are
// few (32 rows of 32 with N 10240, rank 16 13.6 against 13.1; 1000 rows of 300, rank 32
// 175 against 171, rank 48 246 against 247).
inline int lora_expand_waves(int64_t M, int64_t L, int64_t R, int64_t N)
{
    const int64_t tiles = lora_ceil(M, kLoraWindow) * lora_slots(M, L);
    const bool spread = R > 32 || tiles * lora_ceil(N, 256) <= kLoraCus;
    return (M <= 4 || M <= 2 * tiles) && spread ? 1 : 4;
}
// Workgroups of 256 threads of the second product; a launch takes fewer than 2^24.
inline int64_t lora_blocks(int64_t M, int64_t N, int64_t L)
{
    const int64_t windows = lora_ceil(M, kLoraWindow);
    return M <= kLoraFewRows ? windows * lora_slots(M, L) * lora_ceil(N, 256) : windows * lora_ceil(N, 512);
}
int launch_lora(const uint16_t *x, int64_t M, int K, int64_t ldx, const int32_t *index, int64_t L, int R,
                const uint16_t *a, const uint16_t *b, const float *scaling, const int32_t *ranks, int N,
                const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo, float *ws, void *stream);

}  // namespace ck
