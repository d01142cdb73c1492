// Tiled product of e4m3 activations and weights with power-of-two scales for each block
// of 128, on the scaled e4m3 MFMA.
//
//   sums[m, n] = sum_b 2^(sa[m, b] + sw[n / 128, b]) sum_{k in block b} a[m, k] w[n, k]
//
// A block of 128 columns is one 16 x 16 x 128 MFMA, which takes an e8m0 scale for each
// row of either operand: the scales cost no instruction and the sums of all blocks stay
// in one fp32 accumulator.  Weights are the rows of the result (operand A), activations
// its columns: a lane has one row of the output and four neighbouring columns a tile.
//
// A workgroup has kWn x kWm waves, a wave kTn x kTm tiles of 16 x 16.  A stage is one
// block of 128 columns of every row of both operands, 128 bytes a row, moved from
// global memory to LDS directly into two buffers; the 16-byte slots of a row are
// XORed with bits of the row so that the lanes of a fragment's read meet in no bank.
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

__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xc07f); }


template <int kWn_, int kWm_, int kTn_, int kTm_>
struct Tile {
    static constexpr int kWn = kWn_, kWm = kWm_, kTn = kTn_, kTm = kTm_;
    static constexpr int kWaves = kWn * kWm;
    static constexpr int kBn = kWn * kTn * 16, kBm = kWm * kTm * 16;
    static constexpr int kStage = (kBn + kBm) * 128;
    // Scales of 64 steps: a row for each activation row and for two rows of weight blocks.
    static constexpr int kScaleSteps = 64, kScalePitch = kScaleSteps + 4;
    static constexpr int kScales = (kBm + 2) * kScalePitch;
    static constexpr int kPitch = kTn * 32 + 16;      // a staged row of a wave's bf16 tile
    static constexpr int kOut = kWaves * kTm * 16 * kPitch;
    static constexpr int kCodePitch = 128 + 16;       // a staged row of a block's codes
    static constexpr int kCodes = (kBn + 127) / 128 * kBm * kCodePitch;
    static constexpr int kMost = kOut > kCodes ? kOut : kCodes;
    static constexpr int kLds = (2 * kStage > kMost ? 2 * kStage : kMost) + kScales + kWaves * kTm * 16 * 4;
};

template <class T, Fp8Result kKind>
__global__ __launch_bounds__(T::kWaves *kWave) void fp8_tiled_kernel(Fp8Product p, int tiles_m, int tiles_n)
{
    constexpr bool kGated = kKind == Fp8Result::kGated;
    constexpr int kBn = T::kBn, kBm = T::kBm, kTn = T::kTn, kTm = T::kTm, kWaves = T::kWaves;
    static_assert(!kGated || kBn == 256, "a gated tile covers one block of the result");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem_generic[];
    lds_u8 *smem = (lds_u8 *)smem_generic;
    lds_u8 *scales = smem + (2 * T::kStage > T::kMost ? 2 * T::kStage : T::kMost);
    __attribute__((address_space(3))) float *red = (__attribute__((address_space(3))) float *)(scales + T::kScales);

    // Runs of kGroupM tile rows are walked column by column, a contiguous run on each XCD.
    constexpr int kGroupM = 4;
    const int tile = xcd_block(blockIdx.x, tiles_m * tiles_n);
    const int group = tile / (kGroupM * tiles_n);
    const int first_m = group * kGroupM;
    const int group_m = min(kGroupM, tiles_m - first_m);
    const int in_group = tile - group * kGroupM * tiles_n;
    const int64_t m0 = (int64_t)(first_m + in_group % group_m) * kBm;
    const int n0 = (in_group / group_m) * (kGated ? kBn / 2 : kBn);  // first column of the result

    const int t = threadIdx.x, wave = t / kWave, lane = t % kWave;
    const int wn = wave / T::kWm, wm = wave % T::kWm;
    const int l16 = lane % 16, quarter = lane / 16;
    const int K = p.K, steps = (K + 127) / 128;
    const int rows = (int)min((int64_t)kBm, p.M - m0);

    // Operand rows past the end and columns past K read as zero (out of the buffer's range).
    const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(p.a + m0 * p.lda), (short)0, (int)((rows - 1) * p.lda + K), 0x00020000);
    const int w_rows = kGated ? p.I + kBn / 2 : min(kBn, p.N - n0);
    const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(p.w + n0 * p.ldw), (short)0, (int)((w_rows - 1) * p.ldw + K), 0x00020000);
    constexpr int kPast = 0x7fffffff;
    constexpr int kALoads = kBm * 128 / (kWaves * 1024), kWLoads = kBn * 128 / (kWaves * 1024);
    static_assert(kALoads * kWaves * 1024 == kBm * 128 && kWLoads * kWaves * 1024 == kBn * 128, "whole loads");
    // An instruction fills eight rows of a buffer.  Row r of the weights' buffer is row
    // weight_row(r) of the tile's (eight rows stay together).
    auto weight_row = [&](int r) {
        if constexpr (!kGated)
            return r;
        constexpr int kHalf = kTn * 8;   // a wave's rows: half gate, half up
        const int q = r % (2 * kHalf), col = r / (2 * kHalf) * kHalf + q % kHalf;
        return q < kHalf ? col : p.I + col;
    };
    const int swave = __builtin_amdgcn_readfirstlane(wave);
    const int w_lane = lane / 8 * (int)p.ldw, a_lane = lane / 8 * (int)p.lda;
    auto issue = [&](int step, int b) {
        lds_u8 *to = smem + b * T::kStage;
        auto chunk = [&](int eight) { return step * 128 + 16 * swizzle(eight * 8 + lane / 8, lane % 8); };
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) {
            const int eight = swave * kWLoads + i, c = chunk(eight);
            load_lds16(w_rsrc, to + eight * 1024, c < K ? w_lane + c + weight_row(eight * 8) * (int)p.ldw : kPast);
        }
#pragma unroll
        for (int i = 0; i < kALoads; ++i) {
            const int eight = swave * kALoads + i, c = chunk(eight);
            load_lds16(a_rsrc, to + kBn * 128 + eight * 1024, c < K ? a_lane + c + eight * 8 * (int)p.lda : kPast);
        }
    };

    // Scales of steps first .. first + 63 to LDS.
    const uint8_t *sa_tile = p.sa + m0 * p.ldsa;
    const int far = kGated ? p.I / 128 : 1, block_rows = (p.N + 127) / 128;
    auto load_scales = [&](int first) {
        for (int i = t; i < kBm * 16; i += kWaves * kWave) {
            const int r = min(i / 16, rows - 1), b = first + i % 16 * 4;
            if (b < steps)
                *(__attribute__((address_space(3))) uint32_t *)(scales + i / 16 * T::kScalePitch + i % 16 * 4) =
                    *reinterpret_cast<const uint32_t *>(sa_tile + (uint32_t)(r * (int)p.ldsa + b));
        }
        for (int i = t; i < 2 * 64; i += kWaves * kWave) {
            const int r = min(n0 / 128 + i / 64 * far, block_rows - 1), b = min(first + i % 64, steps - 1);
            scales[(kBm + i / 64) * T::kScalePitch + i % 64] = p.sw[(int64_t)r * steps + b];
        }
    };
    load_scales(0);

    issue(0, 0);
    issue(1, 1);

    v4f acc[kTn][kTm];
#pragma unroll
    for (int i = 0; i < kTn; ++i)
#pragma unroll
        for (int j = 0; j < kTm; ++j)
            acc[i][j] = v4f{};

    // Fragment addresses: the swizzle depends on the row's low four bits only, so a wave's
    // tiles differ by constants.
    const int near = 16 * swizzle(l16, quarter), half = 16 * swizzle(l16, quarter + 4);
    const int w_at = (wn * kTn * 16 + l16) * 128, a_at = kBn * 128 + (wm * kTm * 16 + l16) * 128;
    auto fragment = [&](const lds_u8 *row) {
        const u32x4 x = *(lds_u32x4 *)(row + near), y = *(lds_u32x4 *)(row + half);
        return v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    };
    // The block row of a wave's first weight tiles (all of them, unless gated).
    const lds_u8 *sa_at = scales + (wm * kTm * 16 + l16) * T::kScalePitch;
    const lds_u8 *sw_at = scales + (kBm + (kGated ? 0 : wn * kTn * 16 / 128)) * T::kScalePitch;
    uint32_t sa[kTm], sw[2];
    auto read_scales = [&](int kt) {
        const int b = kt % T::kScaleSteps;
        sw[0] = sw_at[b];
        if constexpr (kGated)
            sw[1] = sw_at[T::kScalePitch + b];
#pragma unroll
        for (int j = 0; j < kTm; ++j)
            sa[j] = sa_at[j * 16 * T::kScalePitch + b];
    };

    // One step: a weight tile's fragment is read while the tile before it is multiplied.  The
    // barrier stands before the last tile's products: under them this buffer is filled
    // anew, and the other one's first fragments take the place of those just used.
    v8i a[kTm], w[2];
    auto read_activation = [&](const lds_u8 *stage, int j) { a[j] = fragment(stage + a_at + j * 2048); };
    auto multiply = [&](int i, int j) {
        acc[i][j] = mfma_e4m3<0, 0>(w[i & 1], a[j], acc[i][j], sw[kGated && i >= kTn / 2], sa[j]);
    };
    static_assert(kTn % 2 == 0, "two fragments alternate across steps");
    auto all_but_last = [&](const lds_u8 *stage) {
#pragma unroll
        for (int i = 0; i + 1 < kTn; ++i) {
            w[(i + 1) & 1] = fragment(stage + w_at + (i + 1) * 2048);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kTm; ++j)
                multiply(i, j);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    wait_vmcnt0();
    __syncthreads();
    w[0] = fragment(smem + w_at);
#pragma unroll
    for (int j = 0; j < kTm; ++j)
        read_activation(smem, j);
    for (int first = 0;; first += T::kScaleSteps) {
        const int end = min(first + T::kScaleSteps, steps - 1);   // of the steps that have a successor here
        read_scales(first);
        // One straight run: a load past the last step's columns reads zeros.
        for (int kt = first; kt < end; ++kt) {
            all_but_last(smem + (kt & 1) * T::kStage);
            wait_lgkm0();
            wait_vmcnt0();
            __builtin_amdgcn_s_barrier();
            const lds_u8 *other = smem + (~kt & 1) * T::kStage;
            w[0] = fragment(other + w_at);
            issue(kt + 2, kt & 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kTm; ++j) {
                multiply(kTn - 1, j);
                read_activation(other, j);
                __builtin_amdgcn_sched_barrier(0);
            }
            read_scales(kt + 1);
        }
        if (end < first + T::kScaleSteps)
            break;
        __syncthreads();
        load_scales(end);
        __syncthreads();
    }
    all_but_last(smem + (~steps & 1) * T::kStage);
#pragma unroll
    for (int j = 0; j < kTm; ++j)
        multiply(kTn - 1, j);
    wait_vmcnt0();
    __syncthreads();

    const int64_t mw = m0 + wm * kTm * 16;   // the wave's rows and columns
    // Write the wave's staged bf16 tile: kTm * 16 rows of `cols` columns to dst at column n.
    lds_u8 *mine = smem + wave * kTm * 16 * T::kPitch;
    auto write_bf16 = [&](uint16_t *dst, int64_t ld, int n, int N, int cols_, int from) {
        const int chunks = cols_ / 8, rows_each = kWave / chunks;
        for (int r = lane / chunks; r < kTm * 16; r += rows_each) {
            const int c = lane % chunks;
            const u32x4 v = *(lds_u32x4 *)(mine + r * T::kPitch + from + 16 * c);
            if (mw + r < p.M && n + 8 * c < N)
                *reinterpret_cast<u32x4 *>(dst + (mw + r) * ld + n + 8 * c) = v;
        }
    };
    auto stage_bf16 = [&](int i, int j, const v4f &v) {
        const u32x2 q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        *(__attribute__((address_space(3))) u32x2 *)(mine + (j * 16 + l16) * T::kPitch + (i * 16 + 4 * quarter) * 2) = q;
    };
    // Quantise blocks of 128 columns, each held by kPer waves side by side with kTiles tiles
    // each, and write block i's codes at column n + 128 i, its scales at scale[.. + i].
    auto quantise = [&](const auto &v, auto tiles_c, int n, uint8_t *dst, int64_t ld, uint8_t *scale) {
        constexpr int kTiles = decltype(tiles_c)::value, kPer = 8 / kTiles;
        static_assert(kPer * kTiles == 8 && T::kWn % kPer == 0, "whole blocks");
        constexpr int kBlocks = T::kWn / kPer;
        const int block = wn / kPer, col = wn % kPer * kTiles * 16;
        __syncthreads();  // what the stages or the last blocks held is done with
#pragma unroll
        for (int j = 0; j < kTm; ++j) {
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    a = fmaxf(a, fabsf(v[i][j][r]));
            a = fmaxf(a, __shfl_xor(a, 16));
            a = fmaxf(a, __shfl_xor(a, 32));
            if (quarter == 0)
                red[(wn * T::kWm + wm) * kTm * 16 + j * 16 + l16] = a;
        }
        __syncthreads();
        lds_u8 *to = smem + block * kBm * T::kCodePitch;
#pragma unroll
        for (int j = 0; j < kTm; ++j) {
            float a = 0.f;
#pragma unroll
            for (int o = 0; o < kPer; ++o)
                a = fmaxf(a, red[((block * kPer + o) * T::kWm + wm) * kTm * 16 + j * 16 + l16]);
            const uint32_t s = e8m0_of(a);
            const float inv = e8m0_inverse(s);
            const int row = wm * kTm * 16 + j * 16 + l16;
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
                *(__attribute__((address_space(3))) uint32_t *)(to + row * T::kCodePitch + col + i * 16 + 4 * quarter) =
                    pack_e4m3x4(v[i][j][0] * inv, v[i][j][1] * inv, v[i][j][2] * inv, v[i][j][3] * inv);
            if (wn % kPer == 0 && quarter == 0 && row < rows && n + 128 * block < p.I)
                scale[(m0 + row) * p.ldsq + block] = (uint8_t)s;
        }
        __syncthreads();
        for (int i = t; i < kBlocks * kBm * 8; i += kWaves * kWave) {
            const int row = i / 8 % kBm, b = i / 8 / kBm;
            if (row < rows && n + 128 * b < p.I)
                *reinterpret_cast<u32x4 *>(dst + (m0 + row) * ld + n + 128 * b + i % 8 * 16) =
                    *(lds_u32x4 *)(smem + (b * kBm + row) * T::kCodePitch + i % 8 * 16);
        }
    };

    if constexpr (kKind == Fp8Result::kBf16) {
        const int nw = n0 + wn * kTn * 16;
#pragma unroll
        for (int i = 0; i < kTn; ++i) {
            float b[4] = {0.f, 0.f, 0.f, 0.f};
            if (p.bias)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    b[r] = bf16_to_f32(p.bias[min(nw + i * 16 + 4 * quarter + r, p.N - 1)]);
#pragma unroll
            for (int j = 0; j < kTm; ++j) {
                v4f v = acc[i][j];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[r] += b[r];
                stage_bf16(i, j, v);
            }
        }
        write_bf16(p.out, p.ldo, nw, p.N, kTn * 16, 0);
    } else if constexpr (kGated) {
        constexpr int kHalf = kTn / 2;
        const int col = wn * kHalf * 16;
        if (p.gate_up) {
#pragma unroll
            for (int i = 0; i < kTn; ++i)
#pragma unroll
                for (int j = 0; j < kTm; ++j)
                    stage_bf16(i, j, acc[i][j]);
            write_bf16(p.gate_up, p.ldg, n0 + col, p.I, kHalf * 16, 0);
            write_bf16(p.gate_up + p.I, p.ldg, n0 + col, p.I, kHalf * 16, kHalf * 32);
        }
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
            for (int j = 0; j < kTm; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[i][j][r] = gated(acc[i][j][r], acc[i + kHalf][j][r]);
        quantise(acc, std::integral_constant<int, kHalf>{}, n0, p.q, p.I, p.sq + n0 / 128);
    } else {
        auto gradient = [&](int i, int j, v4f &dg) {   // acc[i][j] becomes du
            const int64_t m = m0 + min(wm * kTm * 16 + j * 16 + l16, rows - 1);
            const int n = min(n0 + wn * kTn * 16 + i * 16, p.I - 16) + 4 * quarter;
            const u32x2 gv = *reinterpret_cast<const u32x2 *>(p.gate_up + m * p.ldg + n);
            const u32x2 uv = *reinterpret_cast<const u32x2 *>(p.gate_up + m * p.ldg + p.I + n);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float g = bf16_to_f32(r % 2 ? gv[r / 2] >> 16 : gv[r / 2] & 0xffffu);
                const float u = bf16_to_f32(r % 2 ? uv[r / 2] >> 16 : uv[r / 2] & 0xffffu);
                const float2 d = gated_gradient(acc[i][j][r], g, u);
                dg[r] = d.x, acc[i][j][r] = d.y;
            }
        };
        v4f dg[kTn][kTm];
#pragma unroll
        for (int i = 0; i < kTn; ++i) {
#pragma unroll
            for (int j = 0; j < kTm; ++j)
                gradient(i, j, dg[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        quantise(dg, std::integral_constant<int, kTn>{}, n0, p.q, 2 * (int64_t)p.I, p.sq + n0 / 128);
        quantise(acc, std::integral_constant<int, kTn>{}, n0, p.q + p.I, 2 * (int64_t)p.I,
                 p.sq + (p.I + n0) / 128);
    }
}

template <class T, Fp8Result kKind>
int launch_tile(const Fp8Product &p, void *stream)
{
    auto kern = fp8_tiled_kernel<T, kKind>;
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
    static_assert(T::kLds <= 160 * 1024, "LDS");
    if (attr != hipSuccess)
        return (int)attr;
    const int tiles_m = (int)((p.M + T::kBm - 1) / T::kBm);
    const int cols = kKind == Fp8Result::kBf16 ? p.N : p.I;
    const int width = kKind == Fp8Result::kGated ? T::kBn / 2 : T::kBn;
    const int tiles_n = (cols + width - 1) / width;
    hipLaunchKernelGGL(kern, dim3((unsigned)tiles_m * (unsigned)tiles_n), dim3(T::kWaves * kWave), T::kLds,
                       reinterpret_cast<hipStream_t>(stream), p, tiles_m, tiles_n);
    return (int)hipGetLastError();
}

using Large = Tile<2, 4, 8, 4>;   // 256 weight rows x 256 activation rows
using Small = Tile<2, 4, 4, 2>;   // 128 x 128

}  // namespace

int launch_fp8_tiled(Fp8Result kind, const Fp8Product &p, void *stream)
{
    switch (kind) {
    case Fp8Result::kBf16:
        return launch_tile<Large, Fp8Result::kBf16>(p, stream);
    case Fp8Result::kGated:
        return launch_tile<Large, Fp8Result::kGated>(p, stream);
    default:
        return launch_tile<Small, Fp8Result::kGrad>(p, stream);
    }
}

}  // namespace ck
