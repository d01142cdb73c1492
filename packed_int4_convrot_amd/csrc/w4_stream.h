// Streaming multiply of packed uint4 expert weights by a few rows, one wave per
// 32 weight rows, on the 32 x 32 x 16 bf16 MFMA.
//
// Per 64-column scale group g,
//   sum_c a_c W[n, c] = s P + (z - 136 s) X,  P = sum a_c (128 + q_c),  X = sum a_c,
// so a group is four MFMAs on bf16(128 + q) (the bit pattern 0x4300 | q: an
// and-or per pair of codes) and two fused multiply-adds per result.  Weight
// rows are the columns of the result, the rows of A its rows: lane l has weight
// row l % 32, and register i of it row 8 (i / 4) + 4 (l / 32) + i % 4 of A, so few
// rows use few registers.
//
// A wave's weights go global -> LDS directly into a ring of its own (no VGPRs, no
// barriers): a stage is four groups, each instruction 128 contiguous bytes of
// eight rows, and one more for the stage's scales and zero points.  (Loads to
// registers in operand order touch 32 rows with 32 bytes each per instruction;
// the address path serialises those, and measured 1.8 TB/s where this form
// measured over twice that.)  The 16-byte slots of a row are XORed with the
// row's low bits, so that the operand reads are free of bank conflicts.
#pragma once

#include "rows_device.h"

namespace ck {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kStageGroups = 4;
constexpr int kStageScales = 4096;               // byte offset of [group][s, z][32 rows] bf16
constexpr int kStageBytes = kStageScales + 512;
constexpr int kStages = 2;
constexpr int kRingBytes = kStages * kStageBytes;

__device__ __forceinline__ v16f mfma32(v8bf a, v8bf b, v16f c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 32 rows of one expert's packed weight [N, 32 G] bytes with scales [G, N]: rows
// n0 .. n0 + 15 and n0 + far .. n0 + far + 15.
__host__ __device__ constexpr int stage_groups(int groups)
{
    return (groups + kStageGroups - 1) / kStageGroups * kStageGroups;
}
struct WeightStream {
    const uint8_t *w;       // this lane's row, of each eight
    const uint16_t *sz;     // this lane's 8 scales or zero points of group 0
    int64_t far_bytes;
    int row_bytes, G, N, slot;
    bool scales;            // this lane loads scales
    lds_u8 *ring;

    __device__ __forceinline__ WeightStream(const uint8_t *packed, const uint16_t *s, const uint16_t *z, int64_t expert,
                                            int rows, int groups, int n0, int far, void *lds)
    {
        const int lane = threadIdx.x % kWave;
        G = groups, N = rows, row_bytes = 32 * groups;
        far_bytes = (int64_t)far * row_bytes;
        w = packed + (expert * rows + n0 + lane / 8) * row_bytes;
        slot = (lane % 8) ^ (lane / 8);
        const int zero_point = lane / 4 % 2, piece = lane % 4;
        scales = lane < 32 && (z || !zero_point);
        sz = (zero_point && z ? z : s) + expert * groups * rows + n0 + piece % 2 * 8 + piece / 2 * far;
        ring = (lds_u8 *)lds;
    }

    // Global -> ring for stage st (groups 4 st .. 4 st + 3; past the row's end the
    // last ones again, which are not used): five instructions.
    __device__ __forceinline__ void issue(int st) const
    {
        lds_u8 *to = ring + st % kStages * kStageBytes;
        const uint8_t *from = w + 16 * min(st * 8 + slot, 2 * G - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_global_load_lds(from + i / 2 * far_bytes + i % 2 * 8 * row_bytes,
                                             (__attribute__((address_space(3))) void *)(to + i * 1024), 16, 0, 0);
        const int g = min(st * kStageGroups + (int)(threadIdx.x % 32) / 8, G - 1);
        if (scales)
            __builtin_amdgcn_global_load_lds(sz + (int64_t)g * N,
                                             (__attribute__((address_space(3))) void *)(to + kStageScales), 16, 0, 0);
    }
};

// Waits for a stage behind which `newer` more have been issued: loads retire in
// order, five instructions a stage.
__device__ __forceinline__ void wait_stage(int newer)
{
    static_assert(kStages <= 4, "vmcnt");
    if (newer >= 3)
        __builtin_amdgcn_s_waitcnt(15 | 0x0F70);
    else if (newer == 2)
        __builtin_amdgcn_s_waitcnt(10 | 0x0F70);
    else if (newer == 1)
        __builtin_amdgcn_s_waitcnt(5 | 0x0F70);
    else
        wait_vmcnt0();
}
// This wave's LDS reads have returned.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// Rows of A in LDS: 16-byte operands [group][4][2 halves][kRows] and group sums
// [group][kRows], with zeros for the groups that fill up the last stage.
template <int kRows>
struct ARows {
    static constexpr int kRegs = kRows <= 2 ? 1 : kRows <= 8 ? 4 : kRows / 2;
    const uint8_t *operands;
    const float *sums;
};

// Stages [st0, st1) of a stream whose first min(kStages, st1 - st0) stages have
// been issued, added to tot; stages up to `last` are issued behind them.  A's
// first group is group a0.
template <int kRows>
__device__ __forceinline__ void stream_stages(const WeightStream &ws, bool zeros, int st0, int st1, int last, int a0,
                                              const ARows<kRows> &A, float (&tot)[ARows<kRows>::kRegs])
{
    constexpr int kRegs = ARows<kRows>::kRegs;
    const int lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32;
    for (int st = st0; st < st1; ++st) {
        wait_stage(min(last - 1 - st, kStages - 1));
        __builtin_amdgcn_sched_barrier(0);
        const lds_u8 *stage = ws.ring + st % kStages * kStageBytes;
        const uint8_t *ap = A.operands + ((st * kStageGroups - a0) * 8 + half) * kRows * 16 + l32 % kRows * 16;
        const float *xp = A.sums + (st * kStageGroups - a0) * kRows + (kRows > 4 ? 4 * half : 0);
        // Straight-line code for the stage's four groups, so that one group's
        // reads and decode overlap another's MFMAs.
#pragma unroll
        for (int u = 0; u < kStageGroups; ++u) {
            const u32x4 w = *(__attribute__((address_space(3))) const u32x4 *)(stage + l32 * 128 +
                                                                              ((2 * u + half) ^ (l32 % 8)) * 16);
            const uint32_t sb =
                *(__attribute__((address_space(3))) const uint16_t *)(stage + kStageScales + u * 128 + l32 * 2);
            const uint32_t zb =
                *(__attribute__((address_space(3))) const uint16_t *)(stage + kStageScales + u * 128 + 64 + l32 * 2);
            v16f acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc = mfma32(*reinterpret_cast<const v8bf *>(ap + (u * 8 + 2 * j) * kRows * 16),
                             w4_bf16_plus128(w[j]), acc);
            const float s = bf16_to_f32(sb);
            const float zc = __builtin_fmaf(-136.f, s, zeros ? bf16_to_f32(zb) : 0.f);
#pragma unroll
            for (int i = 0; i < kRegs; ++i)
                tot[i] = __builtin_fmaf(s, acc[i], __builtin_fmaf(zc, xp[u * kRows + i / 4 * 8 + i % 4], tot[i]));
            if (kRows > 16 || (kRows > 8 && u % 2 == 1))
                __builtin_amdgcn_sched_barrier(0);  // many rows: fewer groups' registers at a time
        }
        if (st + kStages < last) {
            wait_lds();  // the slot's operands have been read
            __builtin_amdgcn_sched_barrier(0);
            ws.issue(st + kStages);
        }
    }
}

// Eight columns into A: operand slot of chunk ch (8 columns) of a row, and the
// group's sum from the eight lanes that hold its chunks.
template <int kRows>
__device__ __forceinline__ void put_chunk(uint8_t *operands, float *sums, int row, int ch, u32x4 v)
{
    const int g = ch / 8, half = ch / 4 % 2, j = ch % 4;
    *reinterpret_cast<u32x4 *>(operands + ((g * 8 + 2 * j + half) * kRows + row) * 16) = v;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        t += bf16_to_f32(v[q] & 0xffffu) + __uint_as_float(v[q] & 0xffff0000u);
#pragma unroll
    for (int b = 1; b < 8; b <<= 1)
        t += __shfl_xor(t, b);
    if (ch % 8 == 0)
        sums[g * kRows + row] = t;
}

// All columns of a stream for kRows rows of A, by every wave of a workgroup of
// kWaves; A goes through LDS in chunks of 16384 / kRows columns.  load(row, ch)
// gives eight columns (chunk ch of the whole row) in operand order; waves that
// are not live only help to load.
constexpr int kChunkElems = 16384;
constexpr int kChunkOperands = kChunkElems * 2, kChunkSums = kChunkElems / 64 * 4;

template <int kRows, int kWaves, class Load>
__device__ __forceinline__ void stream_rows(const WeightStream &ws, bool zeros, bool live, uint8_t *operands,
                                            float *sums, Load &&load, float (&tot)[ARows<kRows>::kRegs])
{
    constexpr int kThreads = kWaves * kWave, kLoads = kChunkElems / 8 / kThreads;
    constexpr int kGroups = kChunkElems / 64 / kRows;  // of a chunk
    static_assert(kGroups % kStageGroups == 0, "a chunk is whole stages");
    const int G = ws.G, last = (G + kStageGroups - 1) / kStageGroups;
    for (int g0 = 0; g0 < G; g0 += kGroups) {
        const int rows_groups = min(kGroups, stage_groups(G) - g0) * kRows;
        u32x4 v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int o = i * kThreads + threadIdx.x;
            const int g = g0 + o / 8 / kRows;
            v[i] = u32x4{0u, 0u, 0u, 0u};
            if (o / 8 < rows_groups && g < G)
                v[i] = load(o / 8 % kRows, g * 8 + o % 8);
        }
        __builtin_amdgcn_sched_barrier(0);  // A's loads before the weights': they retire in order
        if (g0 == 0) {
            if (live)
#pragma unroll
                for (int st = 0; st < kStages; ++st)
                    if (st < last)
                        ws.issue(st);
        }
        __syncthreads();  // the previous chunk has been read
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int o = i * kThreads + threadIdx.x;
            if (o / 8 < rows_groups)
                put_chunk<kRows>(operands, sums, o / 8 % kRows, o / 8 / kRows * 8 + o % 8, v[i]);
        }
        __syncthreads();
        if (live)
            stream_stages<kRows>(ws, zeros, g0 / kStageGroups, min(last, (g0 + kGroups) / kStageGroups), last, g0,
                                 ARows<kRows>{operands, sums}, tot);
    }
}

}  // namespace ck
