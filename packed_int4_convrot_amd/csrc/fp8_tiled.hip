// Tiled product of e4m3 activations and weights with power-of-two scales for each block
// of 128, on the scaled e4m3 MFMA.
//
//   sums[m, n] = sum_b 2^(sa[m, b] + sw[n / 128, b]) sum_{k in block b} a[m, k] w[n, k]
//
// The 32 x 32 x 64 MFMA takes an e8m0 scale for each row of either operand: the scales
// cost no instruction and the sums of all blocks stay in one fp32 accumulator.  (On
// random codes it holds 4.1 PFLOP/s over the chip, the 16 x 16 x 128 one 3.8: both are
// bound by power.)  Weights are the rows of the result (operand A), activations its
// columns: a lane has one row of the output and, of a tile, four times four neighbouring
// columns.
//
// A workgroup has kWn x kWm waves, a wave kTn x kTm tiles of 32 x 32.  A stage is one
// block of 128 columns of every row of both operands, 128 bytes a row, moved from
// global memory to LDS directly into two buffers, four for the small tiles; the 16-byte
// slots of a row are XORed with bits of the row so that the lanes of a fragment's read
// meet in no bank.
//
// What bounds it.  256 x 256 tiles: the matrix cores, 70 % busy over the whole launch at the 1.8 GHz
// that power leaves, and the loads beside them (a step of 1.45 us takes 1.2 with its loads left out):
// 8192 x 10240 x 3840 (rows, K, N) 245 us, 2.6 PFLOP/s, as a large library product here.  Read less
// LDS (four waves of 128 x 128) it takes 2 % more; a burst of loads ahead, prefetches into the L2,
// workgroups that go on to a next tile: none gained.  Small tiles: a step's way through barrier, LDS
// and two products, 0.24 us for 64 x 64.  Eight buffers take as long, and so do steps shared out to
// teams of a workgroup's waves; splitting K over workgroups is what helps.  kGrad's writing of
// results: 4096 rows, H 3840, I 10240 take 23 us less without the reads of g and u, 35 without the
// codes' stores, whatever their order; its tiles fill two and a half rounds of the chip.
//
// kGated: a wave's tiles are half gate rows and half up rows of the same columns, so that
// the activation and the product happen in registers; a workgroup covers the 128
// columns that share a scale of the quantised result.
#include <type_traits>

#include "fp8_device.h"
#include "fp8_launch.h"

namespace ck {
namespace {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;

// LDS slot of 16-byte chunk c of row r, and the reverse.
__device__ __forceinline__ int swizzle(int r, int c) { return c ^ ((r >> 1) & 7); }

// This wave's LDS reads have returned and all but the last N of its loads have landed.
template <int N>
__device__ __forceinline__ void wait_reads_and_loads()
{
    static_assert(N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}

// Registers 8 g .. 8 g + 7 of a lane's row of a 32 x 32 result in bf16: the two lanes of a row exchange
// halves, and this one has columns 16 g + 8 half on.
__device__ __forceinline__ u32x4 bf16x8(const float *v)
{
    uint32_t x0 = pack_bf16x2(v[0], v[1]), x1 = pack_bf16x2(v[2], v[3]);
    uint32_t y0 = pack_bf16x2(v[4], v[5]), y1 = pack_bf16x2(v[6], v[7]);
    swap_halves(x0, y0);
    swap_halves(x1, y1);
    return u32x4{x0, x1, y0, y1};
}

template <int kWn_, int kWm_, int kTn_, int kTm_, int kStages_ = 2>
struct Tile {
    static constexpr int kWn = kWn_, kWm = kWm_, kTn = kTn_, kTm = kTm_, kStages = kStages_;
    static_assert((kStages & (kStages - 1)) == 0, "a power of two");
    static constexpr int kWaves = kWn * kWm;
    static constexpr int kBn = kWn * kTn * 32, kBm = kWm * kTm * 32;
    static constexpr int kStage = (kBn + kBm) * 128;
    // Scales of 64 steps: dwords (four steps) [16][kBm] of the activations, then bytes [2][64]
    // of two rows of weight blocks.
    static constexpr int kScaleSteps = 64, kRowScales = kScaleSteps * kBm;
    static constexpr int kScales = kRowScales + 2 * kScaleSteps;
    static constexpr int kLds = kStages * kStage + kScales + kWaves * 32 * 4;
};

template <class T, Fp8Result kKind>
__global__ __launch_bounds__(T::kWaves *kWave) void fp8_tiled_kernel(Fp8Product p, int tiles_m, int tiles)
{
    constexpr bool kGated = kKind == Fp8Result::kGated;
    constexpr int kBn = T::kBn, kBm = T::kBm, kTn = T::kTn, kTm = T::kTm, kWaves = T::kWaves;
    static_assert(!kGated || kBn == 256, "a gated tile covers one block of the result");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem_generic[];
    lds_u8 *smem = (lds_u8 *)smem_generic;
    lds_u8 *scales = smem + T::kStages * T::kStage;
    __attribute__((address_space(3))) float *red = (__attribute__((address_space(3))) float *)(scales + T::kScales);

    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / kWave), lane = t % kWave;
    const int wn = wave / T::kWm, wm = wave % T::kWm;
    const int l32 = lane % 32, half = lane / 32;
    // Of a split product a workgroup takes blockIdx.y's steps.
    constexpr bool kSplit = kKind == Fp8Result::kSums;
    const int all_steps = (p.K + 127) / 128, step0 = kSplit ? blockIdx.y * p.each : 0;
    const int K = kSplit ? min(p.K - step0 * 128, p.each * 128) : p.K, steps = (K + 127) / 128;

    // Runs of kGroupM tile rows are walked column by column, a contiguous run on each XCD.
    constexpr int kGroupM = 4;
    const int tiles_n = tiles / tiles_m, tile = xcd_block(blockIdx.x, tiles);
    const int group = tile / (kGroupM * tiles_n);
    const int first_m = group * kGroupM;
    const int group_m = min(kGroupM, tiles_m - first_m);
    const int in_group = tile - group * kGroupM * tiles_n;
    const int64_t m0 = (int64_t)(first_m + in_group % group_m) * kBm;     // first row and
    const int n0 = (in_group / group_m) * (kGated ? kBn / 2 : kBn);       // column of the result
    const int rows = (int)min((int64_t)kBm, p.M - m0);
    // Operand rows past the end and columns past K read as zero (out of the buffer's range).
    const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(p.a + m0 * p.lda + step0 * 128), (short)0, (int)((rows - 1) * p.lda + K), 0x00020000);
    const int w_rows = kGated ? p.I + kBn / 2 : min(kBn, p.N - n0);
    const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(p.w + n0 * p.ldw + step0 * 128), (short)0, (int)((w_rows - 1) * p.ldw + K), 0x00020000);
    const __amdgpu_buffer_rsrc_t sa_rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)(p.sa + m0 * p.ldsa + step0), (short)0, (int)(rows * p.ldsa - step0),
                                          0x00020000);
    constexpr int kPast = 0x7fffffff;
    constexpr int kALoads = kBm * 128 / (kWaves * 1024), kWLoads = kBn * 128 / (kWaves * 1024);
    static_assert(kALoads * kWaves * 1024 == kBm * 128 && kWLoads * kWaves * 1024 == kBn * 128, "whole loads");
    // An instruction fills eight rows of a buffer.  Row r of the weights' buffer is row
    // weight_row(r) of the tile's (eight rows stay together).
    auto weight_row = [&](int r) {
        if constexpr (!kGated)
            return r;
        constexpr int kHalf = kTn * 16;   // a wave's rows: half gate, half up
        const int q = r % (2 * kHalf), col = r / (2 * kHalf) * kHalf + q % kHalf;
        return q < kHalf ? col : p.I + col;
    };
    const int w_lane = lane / 8 * (int)p.ldw, a_lane = lane / 8 * (int)p.lda;
    // Load n of a wave's share of a step, into its buffer.  Weight rows are dealt to the waves so
    // that the first half of a wave's loads are of the first half of every wave's tiles.
    constexpr int kEarly = kWLoads / 2, kLate = kWLoads - kEarly;
    static_assert(kWLoads % 2 == 0 && kTn * 2 % kEarly == 0, "halves");
    constexpr int kStages = T::kStages;
    auto buffer = [&](int step) { return smem + (step & (kStages - 1)) * T::kStage; };
    auto issue = [&](int step, bool weights, int n) {
        constexpr int kRows = kTn * 32, kEights = kRows / 16;     // of a wave's tiles; in a half of them
        const int w8 = wave * kEarly + n % kEarly;                // of the early or the late eights
        const int eight = weights ? w8 / kEights * (2 * kEights) + w8 % kEights + n / kEarly * kEights
                                  : wave * kALoads + n;
        const int c = step * 128 + 16 * swizzle(eight * 8 + lane / 8, lane % 8);
        lds_u8 *to = buffer(step) + eight * 1024;
        if (weights)
            load_lds16(w_rsrc, to, c < K ? w_lane + c + weight_row(eight * 8) * (int)p.ldw : kPast);
        else
            load_lds16(a_rsrc, to + kBn * 128, c < K ? a_lane + c + eight * 8 * (int)p.lda : kPast);
    };
    // What is read first of a step: activations and the early weights.
    constexpr int kFirst = kALoads + kEarly, kAll = kFirst + kLate;
    auto issue_first = [&](int step, int n) { issue(step, n >= kALoads, n < kALoads ? n : n - kALoads); };
    auto issue_late = [&](int step, int n) { issue(step, true, kEarly + n); };

    // Scales of steps first .. first + 63 to LDS, a row of the activations in each lane; those of
    // the weights through a register.
    const int far = kGated ? p.I / 128 : 1, block_rows = (p.N + 127) / 128;
    uint32_t sw_in = 0;
    auto load_scales = [&](int first) {
        constexpr int kParts = kBm / kWave, kEach = 16 * kParts / kWaves;
        static_assert(kEach * kWaves == 16 * kParts, "whole loads");
        const int sw_row = min(n0 / 128 + t / 64 % 2 * far, block_rows - 1);
        sw_in = p.sw[(int64_t)sw_row * all_steps + step0 + min(first + t % 64, steps - 1)];
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
            const int e = n * kWaves + wave, part = e % kParts, four = e / kParts;
            if (first + 4 * four < steps)
                load_lds4(sa_rsrc, scales + e % kParts * 256 + four * kBm * 4,
                          min(part * kWave + lane, rows - 1) * (int)p.ldsa + first + 4 * four);
        }
    };
    auto keep_scales = [&]() {
        if (t < 128)
            scales[T::kRowScales + t] = (uint8_t)sw_in;
    };

    // A step has 2 kTn units: the weight tiles in order, two k-halves each.  Two barriers cut it
    // in halves.  Past the first every wave holds all activations and the first half of the
    // weight tiles, past the second the rest: so each part of a buffer is filled for the step
    // after the next as soon as that, and every load has one and a half steps to land.  (With
    // one barrier and one step it takes 792 us for a feed-forward block of 8192 rows, H 3840,
    // I 10240.)  Loads go out one or two at a time between products.
    // Small tiles have more than two buffers: one barrier a step, and loads kStages - 1 steps ahead.
    constexpr int kUnits = 2 * kTn;
    constexpr int kUnderWay = kStages == 2 ? kAll : (kStages - 2) * kAll;   // at a barrier
    auto first_loads = [&]() {
        load_scales(0);
#pragma unroll
        for (int step = 0; step < kStages - 1; ++step) {
#pragma unroll
            for (int n = 0; n < kFirst; ++n)
                issue_first(step, n);
#pragma unroll
            for (int n = 0; n < kLate; ++n)
                issue_late(step, n);
        }
        if constexpr (kStages == 2)
#pragma unroll
            for (int n = 0; n < kFirst; ++n)
                issue_first(1, n);
    };
    // Loads under unit u of a step.
    auto issue_under = [&](int kt, int u) {
        if constexpr (kStages > 2) {
            constexpr int kSlots = kUnits - 1;
#pragma unroll
            for (int n = u * kAll / kSlots; n < (u + 1) * kAll / kSlots; ++n)
                n < kFirst ? issue_first(kt + kStages - 1, n) : issue_late(kt + kStages - 1, n - kFirst);
        } else if (u < kTn - 1) {
#pragma unroll
            for (int n = u * kLate / (kTn - 1); n < (u + 1) * kLate / (kTn - 1); ++n)
                issue_late(kt + 1, n);
        } else {
#pragma unroll
            for (int n = (u - kTn + 1) * kFirst / kTn; n < (u - kTn + 2) * kFirst / kTn; ++n)
                issue_first(kt + 2, n);
        }
    };

    v16f acc[kTn][kTm];

    // A lane's fragment of k-half s: 32 bytes from 64 s + 32 half on, two slots.  The swizzle
    // depends on the row's low four bits only, so a wave's tiles differ by constants.
    const int slot0 = 16 * swizzle(l32, 2 * half), slot1 = 16 * swizzle(l32, 2 * half + 1);
    const int w_at = (wn * kTn * 32 + l32) * 128, a_at = kBn * 128 + (wm * kTm * 32 + l32) * 128;
    auto fragment = [&](const lds_u8 *row, int s) {   // chunk + 4 is slot ^ 64
        const u32x4 x = *(lds_u32x4 *)(row + (slot0 ^ (64 * s))), y = *(lds_u32x4 *)(row + (slot1 ^ (64 * s)));
        return v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    };
    // The block row of a wave's first weight tiles (all of them, unless gated).
    const lds_u8 *sa_at = scales + (wm * kTm * 32 + l32) * 4;
    const lds_u8 *sw_at = scales + T::kRowScales + (kGated ? 0 : wn * kTn * 32 / 128) * T::kScaleSteps;
    uint32_t sa[kTm], sw[2], sa_next[kTm], sw_next[2];
    auto read_scales = [&](int kt) {
        const int b = kt % T::kScaleSteps;
        sw_next[0] = sw_at[b];
        if constexpr (kGated)
            sw_next[1] = sw_at[T::kScaleSteps + b];
#pragma unroll
        for (int j = 0; j < kTm; ++j)
            sa_next[j] = sa_at[j * 32 * 4 + b / 4 * kBm * 4 + b % 4];
    };
    auto take_scales = [&]() {
        sw[0] = sw_next[0];
        if constexpr (kGated)
            sw[1] = sw_next[1];
#pragma unroll
        for (int j = 0; j < kTm; ++j)
            sa[j] = sa_next[j];
    };

    // A unit's weight fragment is read while the unit before it is multiplied; the barriers stand
    // before the last unit's products of either half, under which the next half's first
    // fragments are read.
    v8i a[2][kTm], w[2];
    auto multiply = [&](int u, int j) {
        const int i = u / 2, s = u % 2;
        acc[i][j] = mfma_e4m3(w[u & 1], a[s][j], acc[i][j], sw[kGated && i >= kTn / 2], sa[j]);
    };
    auto all_but_last = [&](int kt) {
        const lds_u8 *stage = buffer(kt);
#pragma unroll
        for (int u = 0; u + 1 < kUnits; ++u) {
            if (kStages == 2 && u == kTn - 1) {
                wait_reads_and_loads<kUnderWay>();
                __builtin_amdgcn_s_barrier();
            }
            w[(u + 1) & 1] = fragment(stage + w_at + (u + 1) / 2 * 4096, (u + 1) % 2);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kTm; ++j)
                multiply(u, j);
            issue_under(kt, u);
            if (u == kUnits - 2)
                read_scales(kt + 1);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Results.  A lane has row 32 j + l32 of the wave's and, in registers 4 q .. 4 q + 3 of tile i,
    // its columns from 32 i + 8 q + 4 half on.  The two lanes of a row exchange halves, so that
    // each has 16 bytes that lie together.
    // Columns 32 i + 16 h .. of a tile's codes, h = half.
    auto codes16 = [&](const float(&v)[16], float scale) {
        uint32_t c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            c[q] = pack_e4m3x4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3], scale);
        swap_halves(c[0], c[2]);
        swap_halves(c[1], c[3]);
        return u32x4{c[0], c[2], c[1], c[3]};
    };
    // The reverse of bf16x8, to fp32.
    auto floats8 = [&](u32x4 x, float *v) {
        uint32_t d[4] = {x[0], x[1], x[2], x[3]};
        swap_halves(d[0], d[2]);
        swap_halves(d[1], d[3]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] = r % 2 ? __uint_as_float(d[r / 2] & 0xffff0000u) : bf16_to_f32(d[r / 2] & 0xffffu);
            v[4 + r] = r % 2 ? __uint_as_float(d[2 + r / 2] & 0xffff0000u) : bf16_to_f32(d[2 + r / 2] & 0xffffu);
        }
    };
    // Quantise a row's kTiles tiles, the largest of which is a, with the waves that hold the other
    // columns of its block of 128: the scale, and the codes of tile(i) at column n + 32 i.
    auto quantise = [&](auto tiles, float a, auto tile, int m, int n, uint8_t *dst, uint8_t *scale) {
        constexpr int kTiles = decltype(tiles)::value, kPer = 4 / kTiles;   // waves of a block
        static_assert(kPer * kTiles == 4 && T::kWn % kPer == 0, "whole blocks");
        a = fmaxf(a, __shfl_xor(a, 32));
        if constexpr (kPer > 1) {
            if (half == 0)
                red[wave * 32 + l32] = a;
            lds_barrier();
#pragma unroll
            for (int o = 0; o < kPer; ++o)
                a = fmaxf(a, red[((wn / kPer * kPer + o) * T::kWm + wm) * 32 + l32]);
            lds_barrier();   // read before the next row's is written
        }
        const uint32_t s = e8m0_of(a);
        const float by = e8m0_value(s);
        const bool inside = m < rows && n < p.I;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            float v[16];
            tile(i, v);
            const u32x4 c = codes16(v, by);
            if (inside)
                *reinterpret_cast<u32x4 *>(dst + 32 * i + 16 * half) = c;
        }
        if (wn % kPer == 0 && half == 0 && inside)
            *scale = (uint8_t)s;
    };
    // bf16 rows go through the wave's part of the stages, whose 16-byte slots are XORed with the
    // row, so that a store writes four whole rows of the wave's columns.
    constexpr int kRowBytes = kTn * 64, kSlots = kRowBytes / 16;
    lds_u8 *mine = smem + wave * kTm * 32 * kRowBytes;
    auto stage_bf16 = [&](int i, int j, int g, const float *v) {
        const int r = j * 32 + l32, slot = 4 * i + 2 * g + half;
        *(__attribute__((address_space(3))) u32x4 *)(mine + r * kRowBytes + 16 * (slot ^ (r % kSlots))) = bf16x8(v);
    };
    // Slots `from` .. `from` + `width` - 1 of the staged rows to dst, column n.
    auto write_bf16 = [&](uint16_t *dst, int64_t ld, int n, int N, auto width, int from) {
        constexpr int kWidth = decltype(width)::value, kRows = kWave / kWidth;
#pragma unroll
        for (int r0 = 0; r0 < kTm * 32; r0 += kRows) {
            const int r = r0 + lane / kWidth, c = lane % kWidth, m = wm * kTm * 32 + r;
            const u32x4 v = *(lds_u32x4 *)(mine + r * kRowBytes + 16 * ((from + c) ^ (r % kSlots)));
            if (m < rows && n + 8 * c < N)
                *reinterpret_cast<u32x4 *>(dst + (m0 + m) * ld + n + 8 * c) = v;
        }
    };
    static_assert(kKind != Fp8Result::kGrad || kWaves * kTn * 4 * kWave * 16 <= kStages * T::kStage, "du fits the stages");

    const int nw = n0 + wn * (kGated ? kTn / 2 : kTn) * 32;   // the wave's first column
    // kGrad reads a tile's g and u while the one before is worked on, the first under the last step
    // of large tiles (2000 rows, H 1024, I 4096: 50.9 us, each at its time 54.0; 1024 rows, H 2048, I
    // 5120: 56.4, 58.8; 77 rows, H 2112, I 1280: 21.9 also under a small tile's, 21.5 after).
    constexpr int kAhead = kKind == Fp8Result::kGrad ? 1 : 0;
    u32x4 kept[kAhead + 1][4];
    auto load_piece = [&](int piece) {
        const int m = wm * kTm * 32 + piece / kTn * 32 + l32;
        const uint16_t *g = p.gate_up + (m0 + min(m, rows - 1)) * p.ldg + (nw < p.I ? nw : p.I - kTn * 32) +
                            piece % kTn * 32 + 8 * half;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            kept[piece % (kAhead + 1)][x] = *reinterpret_cast<const u32x4 *>(g + x / 2 * p.I + x % 2 * 16);
    };

    first_loads();
#pragma unroll
    for (int i = 0; i < kTn; ++i)
#pragma unroll
        for (int j = 0; j < kTm; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][j][r] = 0.f;
    keep_scales();
    wait_reads_and_loads<kStages == 2 ? kFirst : (kStages - 2) * kAll>();   // the first step is there
    lds_barrier();
    w[0] = fragment(smem + w_at, 0);
#pragma unroll
    for (int j = 0; j < kTm; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s)
            a[s][j] = fragment(smem + a_at + j * 4096, s);
    for (int first = 0;; first += T::kScaleSteps) {
        const int end = __builtin_amdgcn_readfirstlane(min(first + T::kScaleSteps, steps - 1));
        read_scales(first);
        take_scales();
        // One straight run: a load past the last step's columns reads zeros.
        for (int kt = first; kt < end; ++kt) {
            all_but_last(kt);
            wait_reads_and_loads<kUnderWay>();
            __builtin_amdgcn_s_barrier();
            const lds_u8 *other = buffer(kt + 1);
            w[0] = fragment(other + w_at, 0);
#pragma unroll
            for (int j = 0; j < kTm; ++j)
                a[0][j] = fragment(other + a_at + j * 4096, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kTm; ++j) {
                multiply(kUnits - 1, j);
                a[1][j] = fragment(other + a_at + j * 4096, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            take_scales();
        }
        if (end < first + T::kScaleSteps)
            break;
        lds_barrier();
        load_scales(end);
        keep_scales();
        wait_vmcnt0();
        lds_barrier();
    }
    if constexpr (kKind == Fp8Result::kGrad && kStages == 2)
        load_piece(0);
    all_but_last(steps - 1);
#pragma unroll
    for (int j = 0; j < kTm; ++j)
        multiply(kUnits - 1, j);
    // All products are done here: left to itself the compiler takes some of the last step's, and
    // the fragments that they need, into the writing of the results.
#pragma unroll
    for (int i = 0; i < kTn; ++i)
#pragma unroll
        for (int j = 0; j < kTm; ++j)
            asm volatile("" : "+v"(acc[i][j]));
    wait_vmcnt0();   // loads past the last step
    lds_barrier();

    if constexpr (kSplit) {
        v4f *to = reinterpret_cast<v4f *>(p.sums) + lane +
                  (((int64_t)blockIdx.y * tiles + m0 / kBm * tiles_n + n0 / kBn) * kWaves + wave) * kTn * kTm * 4 * kWave;
#pragma unroll
        for (int i = 0; i < kTn; ++i)
#pragma unroll
            for (int j = 0; j < kTm; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v16f &x = acc[i][j];
                    to[((i * kTm + j) * 4 + q) * kWave] = v4f{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
                }
        return;
    }
    if (kKind == Fp8Result::kBf16 || (kGated && p.gate_up)) {
#pragma unroll
        for (int i = 0; i < kTn; ++i)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float b[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    b[r] = 0.f;
                if (kKind == Fp8Result::kBf16 && p.bias)
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        b[r] = bf16_to_f32(
                            p.bias[min(nw + i * 32 + 16 * g + r / 4 * 8 + 4 * half + r % 4, p.N - 1)]);
#pragma unroll
                for (int j = 0; j < kTm; ++j) {
                    float v[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        v[r] = acc[i][j][8 * g + r] + b[r];
                    stage_bf16(i, j, g, v);
                }
            }
        if constexpr (kKind == Fp8Result::kBf16) {
            write_bf16(p.out, p.ldo, nw, p.N, std::integral_constant<int, kSlots>{}, 0);
        } else {
            const std::integral_constant<int, kSlots / 2> width;
            write_bf16(p.gate_up, p.ldg, nw, p.I, width, 0);
            write_bf16(p.gate_up + p.I, p.ldg, nw, p.I, width, kSlots / 2);
        }
    }
    if constexpr (kKind == Fp8Result::kGrad && kStages > 2)
        load_piece(0);
#pragma unroll
    for (int j = 0; j < (kKind == Fp8Result::kBf16 ? 0 : kTm); ++j) {
        const int m = wm * kTm * 32 + j * 32 + l32;
        const int64_t row = m0 + m;
        if constexpr (kGated) {
            constexpr int kHalf = kTn / 2;
            float h[kHalf][16], largest = 0.f;
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    h[i][r] = gated(acc[i][j][r], acc[i + kHalf][j][r]);
                    largest = fmaxf(largest, fabsf(h[i][r]));
                }
            quantise(std::integral_constant<int, kHalf>{}, largest,
                     [&](int i, float *v) {
#pragma unroll
                         for (int r = 0; r < 16; ++r)
                             v[r] = h[i][r];
                     },
                     m, nw, p.q + row * p.I + nw, p.sq + row * p.ldsq + nw / 128);
        } else if constexpr (kKind == Fp8Result::kGrad) {
            // dg stays in registers, du waits in the wave's part of the stages.
            lds_u8 *wait = smem + (wave * kTn * 4 * kWave + lane) * 16;
            float dg[kTn][16], largest_g = 0.f, largest_u = 0.f;
#pragma unroll
            for (int i = 0; i < kTn; ++i) {
                const int piece = j * kTn + i;
                if (piece + kAhead < kTm * kTn)
                    load_piece(piece + kAhead);
#pragma unroll
                for (int g2 = 0; g2 < 2; ++g2) {
                    __builtin_amdgcn_sched_barrier(0);
                    float g[8], u[8];
                    floats8(kept[piece % (kAhead + 1)][g2], g);
                    floats8(kept[piece % (kAhead + 1)][2 + g2], u);
                    v4f du[2];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float2 d = gated_gradient(acc[i][j][8 * g2 + r], g[r], u[r]);
                        dg[i][8 * g2 + r] = d.x, du[r / 4][r % 4] = d.y;
                        largest_g = fmaxf(largest_g, fabsf(d.x)), largest_u = fmaxf(largest_u, fabsf(d.y));
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        *(__attribute__((address_space(3))) v4f *)(wait + (i * 4 + 2 * g2 + q) * kWave * 16) = du[q];
                }
            }
            uint8_t *to = p.q + row * 2 * p.I + nw, *scale = p.sq + row * p.ldsq + nw / 128;
            const std::integral_constant<int, kTn> tiles_c;
            quantise(tiles_c, largest_g,
                     [&](int i, float *v) {
#pragma unroll
                         for (int r = 0; r < 16; ++r)
                             v[r] = dg[i][r];
                     },
                     m, nw, to, scale);
            quantise(tiles_c, largest_u,
                     [&](int i, float *v) {
#pragma unroll
                         for (int q = 0; q < 4; ++q) {
                             const v4f d = *(__attribute__((address_space(3))) v4f *)(wait + (i * 4 + q) * kWave * 16);
#pragma unroll
                             for (int r = 0; r < 4; ++r)
                                 v[4 * q + r] = d[r];
                         }
                     },
                     m, nw, to + p.I, scale + p.I / 128);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Adds a split product's sums in the order of its splits.  A wave has a 32 x 32 tile of the result.
template <class T>
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8Product p, int splits, int tiles, int tiles_n)
{
    const int lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32;
    constexpr int kEach = T::kTn * T::kTm;   // of a wave's; kEach * kWaves of a workgroup's
    const int w = blockIdx.x * 4 + threadIdx.x / kWave, tile = w / (kEach * T::kWaves);
    const int wave = w / kEach % T::kWaves, i = w % kEach / T::kTm, j = w % T::kTm;
    const int64_t m = (int64_t)(tile / tiles_n) * T::kBm + (wave % T::kWm * T::kTm + j) * 32 + l32;
    const int n = tile % tiles_n * T::kBn + (wave / T::kWm * T::kTn + i) * 32;
    const v4f *from = reinterpret_cast<const v4f *>(p.sums) + (int64_t)w * 4 * kWave + lane;
    float s[16];
#pragma unroll
    for (int r = 0; r < 16; ++r)
        s[r] = 0.f;
#pragma unroll 2
    for (int z = 0; z < splits; ++z)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const v4f x = from[((int64_t)z * tiles * T::kWaves * kEach * 4 + q) * kWave];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s[4 * q + r] += x[r];
        }
    if (p.bias)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            s[r] += bf16_to_f32(p.bias[min(n + r / 4 * 8 + 4 * half + r % 4, p.N - 1)]);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const u32x4 x = bf16x8(s + 8 * g);
        const int c = n + 16 * g + 8 * half;
        if (m < p.M && c < p.N)
            *reinterpret_cast<u32x4 *>(p.out + m * p.ldo + c) = x;
    }
}

template <class T, Fp8Result kKind>
int launch_tile(const Fp8Product &p, int64_t splits, void *stream)
{
    auto kern = fp8_tiled_kernel<T, kKind>;
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
    static_assert(T::kLds <= 160 * 1024, "LDS");
    if (attr != hipSuccess)
        return (int)attr;
    const int64_t tiles_m = (p.M + T::kBm - 1) / T::kBm;
    const int cols = kKind == Fp8Result::kGated || kKind == Fp8Result::kGrad ? p.I : p.N;
    const int width = kKind == Fp8Result::kGated ? T::kBn / 2 : T::kBn;
    const int64_t tiles = tiles_m * ((cols + width - 1) / width);
    hipLaunchKernelGGL(kern, dim3((unsigned)tiles, (unsigned)splits), dim3(T::kWaves * kWave), T::kLds,
                       reinterpret_cast<hipStream_t>(stream), p, (int)tiles_m, (int)tiles);
    const int e = (int)hipGetLastError();
    if constexpr (kKind == Fp8Result::kSums) {
        if (e != 0)
            return e;
        hipLaunchKernelGGL(fp8_join_kernel<T>, dim3((unsigned)(tiles * T::kWaves * T::kTn * T::kTm / 4)),
                           dim3(256), 0,
                           reinterpret_cast<hipStream_t>(stream), p, (int)splits, (int)tiles, (int)(tiles / tiles_m));
        return (int)hipGetLastError();
    }
    return e;
}

// The three smallest tiles, split or not.
template <class T>
int launch_small(const Fp8Product &p, const Fp8Plan &plan, float *sums, void *stream)
{
    if (plan.splits == 1)
        return launch_tile<T, Fp8Result::kBf16>(p, 1, stream);
    Fp8Product part = p;
    part.each = (int)plan.each, part.sums = sums;
    return launch_tile<T, Fp8Result::kSums>(part, plan.splits, stream);
}

template <Fp8Result kKind>
int launch_kind(const Fp8Product &p, const Fp8Plan &plan, float *sums, void *stream)
{
    constexpr bool kGated = kKind == Fp8Result::kGated, kGrad = kKind == Fp8Result::kGrad;
    using Narrow = Tile<4, 2, 1, 1, 4>;
    switch (plan.tile) {
    case Fp8Tile::k256x256:
        return launch_tile<Tile<2, 4, 4, 2>, kKind>(p, 1, stream);
    case Fp8Tile::k256x192:
        return launch_tile<Tile<4, 2, 2, 3>, kKind>(p, 1, stream);
    case Fp8Tile::k256x128:
        return launch_tile<Tile<4, 2, 2, 2>, kKind>(p, 1, stream);
    case Fp8Tile::k256x64:
        if constexpr (kGated)
            return launch_tile<Tile<4, 2, 2, 1>, kKind>(p, 1, stream);
        break;
    case Fp8Tile::k128x128:
        if constexpr (kGrad)
            return launch_tile<Tile<2, 4, 2, 1, 4>, kKind>(p, 1, stream);
        else if constexpr (!kGated)
            return launch_small<Tile<2, 4, 2, 1, 4>>(p, plan, sums, stream);
        break;
    case Fp8Tile::k128x64:
        if constexpr (kGrad)
            return launch_tile<Narrow, kKind>(p, 1, stream);
        else if constexpr (!kGated)
            return launch_small<Narrow>(p, plan, sums, stream);
        break;
    case Fp8Tile::k64x64:
        if constexpr (kKind == Fp8Result::kBf16)
            return launch_small<Tile<2, 2, 1, 1, 4>>(p, plan, sums, stream);
        break;
    }
    return (int)hipErrorInvalidValue;
}

}  // namespace

int launch_fp8_tiled(Fp8Result kind, const Fp8Product &p, const Fp8Plan &plan, float *sums, void *stream)
{
    switch (kind) {
    case Fp8Result::kBf16:
        return launch_kind<Fp8Result::kBf16>(p, plan, sums, stream);
    case Fp8Result::kGated:
        return launch_kind<Fp8Result::kGated>(p, plan, sums, stream);
    case Fp8Result::kGrad:
        return launch_kind<Fp8Result::kGrad>(p, plan, sums, stream);
    default:
        return (int)hipErrorInvalidValue;
    }
}

}  // namespace ck
