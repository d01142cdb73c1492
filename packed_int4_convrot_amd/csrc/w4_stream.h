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
// the address path serialises those: 64 tokens of 8 in 128 experts took 578 us that
// way and 346 us in the first form of this one.)  The 16-byte slots of a row are XORed with the
// row's low bits, so that the lanes of an operand read meet in no bank (all LDS
// instructions of the many-pair products together: 0.6 conflict cycles each).
//
// The codes' offset makes P and X sums that largely cancel: terms of 128 + q where the
// weight has q - 8, some 30 times its size.  In fp32 that leaves an error of about 2^-19
// of a result, far below its last rounding, and it bounds the activations' range.
#pragma once

#include "gemv_reduce.h"
#include "rows_device.h"

namespace ck {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kStageGroups = 4;
constexpr int kStageScales = 4096;               // byte offset of [group][s, z][32 rows] bf16
constexpr int kStageBytes = kStageScales + 512;
constexpr int kStages = 2;                       // of a ring, unless a kernel asks for more
constexpr int kRingBytes = kStages * kStageBytes;

__device__ __forceinline__ v16f mfma32(v8bf a, v8bf b, v16f c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__host__ __device__ constexpr int stage_groups(int groups)
{
    return (groups + kStageGroups - 1) / kStageGroups * kStageGroups;
}

// Packed weights [experts][N, 32 row_groups] bytes with scales [experts][row_groups,
// N], read by tiles of 32 "rows" of one expert: 16 from row n0 on and 16 far
// ones, which are either rows far away (gate and up) or the second half of the
// same rows' columns.  A cursor says which stages to read: next() sets the tile of
// the next stage and its number, or returns false at the end.
template <int kDepth = kStages>
struct WeightStream {
    const uint8_t *packed, *w;      // w, sz: this lane's row of each eight, and its
    const uint16_t *s, *z, *sz;     // 8 scales or zero points of group 0, in the tile
    int64_t far_bytes, far_scale;
    int row_bytes, row_groups, N, slot;
    int G, far_G;                   // groups of the near and the far rows
    int place, use;                 // ring slots of the next to issue and to consume
    int ahead;                      // stages issued and not consumed
    bool scales, zero_point;        // this lane loads scales; they are zero points
    lds_u8 *ring;

    // far > 0: the far rows are `far` rows on; 0: column halves.
    __device__ __forceinline__ WeightStream(const uint8_t *packed_, const uint16_t *s_, const uint16_t *z_, int rows,
                                            int groups, int far, void *lds)
    {
        const int lane = threadIdx.x % kWave;
        packed = packed_, s = s_, z = z_, N = rows, row_groups = groups, row_bytes = 32 * groups;
        if (far > 0) {
            G = far_G = groups;
            far_bytes = (int64_t)far * row_bytes, far_scale = far;
        } else {
            G = (groups + 1) / 2, far_G = groups - G;
            far_bytes = (int64_t)G * 32, far_scale = (int64_t)G * rows;
            if (far_G == 0)  // a single group: the far rows meet zeros
                far_G = G, far_bytes = far_scale = 0;
        }
        slot = (lane % 8) ^ (lane / 8);
        zero_point = lane / 4 % 2;
        scales = lane < 32 && (z || !zero_point);
        ring = (lds_u8 *)lds;
        place = use = ahead = 0;
    }
    __device__ __forceinline__ void tile(int expert, int n0)
    {
        const int lane = threadIdx.x % kWave, piece = lane % 4;
        w = packed + ((int64_t)expert * N + n0 + lane / 8) * row_bytes;
        sz = (zero_point && z ? z : s) + (int64_t)expert * row_groups * N + n0 + piece % 2 * 8 +
             piece / 2 * far_scale;
    }
    __device__ __forceinline__ int stages() const { return (G + kStageGroups - 1) / kStageGroups; }
    // Global -> ring for one stage of the tile (past the row's end the last columns
    // again, which meet zeros): five instructions.
    __device__ __forceinline__ void issue(int stage)
    {
        lds_u8 *to = ring + place * kStageBytes;
        const uint8_t *near = w + 16 * min(stage * 8 + slot, 2 * G - 1);
        const uint8_t *far = w + far_bytes + 16 * min(stage * 8 + slot, 2 * far_G - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_global_load_lds((i < 2 ? near : far) + i % 2 * 8 * row_bytes,
                                             (__attribute__((address_space(3))) void *)(to + i * 1024), 16, 0, 0);
        const int lane = threadIdx.x % kWave;
        const int g = min(stage * kStageGroups + lane % 32 / 8, (lane % 4 < 2 ? G : far_G) - 1);
        if (scales)
            __builtin_amdgcn_global_load_lds(sz + (int64_t)g * N,
                                             (__attribute__((address_space(3))) void *)(to + kStageScales), 16, 0, 0);
        place = place + 1 == kDepth ? 0 : place + 1;
        ++ahead;
    }
    template <class Cursor>
    __device__ __forceinline__ void start(Cursor &cursor)
    {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            int stage;
            if (cursor.next(*this, stage))
                issue(stage);
        }
    }
};

// Cursor over stages [st, end) of the tile that is set.
struct OneTile {
    int st, end;
    template <class Stream>
    __device__ __forceinline__ bool next(Stream &, int &stage)
    {
        stage = st;
        return st++ < end;
    }
};

// Waits for a stage behind which `newer` more have been issued, and at least
// `stores` (0, 2, 4 or 8) vector stores: they retire in order, five instructions a
// stage.  A count that is too low only waits for more.
template <int kCount>
__device__ __forceinline__ void wait_vmcnt_n()
{
    static_assert(kCount < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((kCount & 15) | (kCount >> 4 << 14) | 0x0F70);
}
template <int kNewer>
__device__ __forceinline__ void wait_behind(int stores)
{
    if (stores >= 8)
        wait_vmcnt_n<5 * kNewer + 8>();
    else if (stores >= 4)
        wait_vmcnt_n<5 * kNewer + 4>();
    else if (stores >= 2)
        wait_vmcnt_n<5 * kNewer + 2>();
    else
        wait_vmcnt_n<5 * kNewer>();
}
__device__ __forceinline__ void wait_stage(int newer, int stores)
{
    if (newer >= 2)
        wait_behind<2>(stores);
    else if (newer == 1)
        wait_behind<1>(stores);
    else
        wait_behind<0>(stores);
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

// Stages [st0, st1) of a tile, the stream's next to consume, added to tot; the
// cursor's next stages are issued behind them.  A's first group is group a0.
// after_first() runs between the first stage's reads and the issue behind it and
// returns how many vector stores it issued at least: the next stage is older than
// they are, so the wait for it lets them be outstanding.
template <int kRows, int kDepth, class Cursor, class Hook>
__device__ __forceinline__ void stream_stages(WeightStream<kDepth> &ws, Cursor &cursor, bool zeros, int st0, int st1,
                                              int a0, const ARows<kRows> &A, float (&tot)[ARows<kRows>::kRegs],
                                              Hook &&after_first)
{
    static_assert(kDepth <= 3, "wait_stage");
    constexpr int kRegs = ARows<kRows>::kRegs;
    const int lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32;
    int stores = 0;
    for (int st = st0; st < st1; ++st) {
        // With more than two stages in flight the stores would be behind several.
        wait_stage(ws.ahead - 1, kDepth == 2 ? stores : 0);
        stores = 0;
        __builtin_amdgcn_sched_barrier(0);
        const lds_u8 *stage = ws.ring + ws.use * kStageBytes;
        ws.use = ws.use + 1 == kDepth ? 0 : ws.use + 1;
        --ws.ahead;
        // The stage into registers first, so that the next one can be issued into
        // its slot before the multiplication.
        u32x4 w[kStageGroups];
        uint32_t sb[kStageGroups], zb[kStageGroups];
#pragma unroll
        for (int u = 0; u < kStageGroups; ++u) {
            w[u] = *(__attribute__((address_space(3))) const u32x4 *)(stage + l32 * 128 +
                                                                     ((2 * u + half) ^ (l32 % 8)) * 16);
            sb[u] = *(__attribute__((address_space(3))) const uint16_t *)(stage + kStageScales + u * 128 + l32 * 2);
            zb[u] = *(__attribute__((address_space(3))) const uint16_t *)(stage + kStageScales + u * 128 + 64 + l32 * 2);
        }
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        if (st == st0)
            stores = after_first();
        int next;
        if (cursor.next(ws, next))
            ws.issue(next);
        __builtin_amdgcn_sched_barrier(0);
        // Straight-line code for the stage's four groups, so that one group's
        // reads and decode overlap another's MFMAs.
        const uint8_t *ap = A.operands + ((st * kStageGroups - a0) * 8 + half) * kRows * 16 + l32 % kRows * 16;
        const float *xp = A.sums + (st * kStageGroups - a0) * kRows + (kRows > 4 ? 4 * half : 0);
#pragma unroll
        for (int u = 0; u < kStageGroups; ++u) {
            v16f acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc = mfma32(*reinterpret_cast<const v8bf *>(ap + (u * 8 + 2 * j) * kRows * 16),
                             w4_bf16_plus128(w[u][j]), acc);
            const float s = bf16_to_f32(sb[u]);
            const float zc = __builtin_fmaf(-136.f, s, zeros ? bf16_to_f32(zb[u]) : 0.f);
#pragma unroll
            for (int i = 0; i < kRegs; ++i)
                tot[i] = __builtin_fmaf(s, acc[i], __builtin_fmaf(zc, xp[u * kRows + i / 4 * 8 + i % 4], tot[i]));
            if (kRows > 8 && u % 2 == 1)
                __builtin_amdgcn_sched_barrier(0);  // many rows: fewer groups' registers at a time
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
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t pair = v[q];  // times (1, 1)
        t = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, pair), __builtin_bit_cast(v2bf, 0x3F803F80u), t,
                                            false);
    }
    t += __uint_as_float(lane_xor_u<1>(__float_as_uint(t)));
    t += __uint_as_float(lane_xor_u<2>(__float_as_uint(t)));
    t += __uint_as_float(lane_mirror8_u(__float_as_uint(t)));
    if (ch % 8 == 0)
        sums[g * kRows + row] = t;
}

// A for a workgroup of kWaves waves, in LDS: whole where it fits, else in chunks
// of 32768 / kRows columns.  load(row, chunk of 8 columns) gives columns in operand
// order.  started() runs first: weights issued there arrive before A, whose
// loads' wait covers them.
constexpr int kChunkElems = 32768;
constexpr int kChunkOperands = kChunkElems * 2, kChunkSums = kChunkElems / 64;

template <int kRows, int kWaves, class Load, class Started>
__device__ __forceinline__ void fill_rows(int G, int g0, uint8_t *operands, float *sums, Load &&load, Started &&started)
{
    constexpr int kThreads = kWaves * kWave, kLoads = kChunkElems / 8 / kThreads;
    constexpr int kGroups = kChunkElems / 64 / kRows;  // of a chunk
    static_assert(kGroups % kStageGroups == 0, "a chunk is whole stages");
    const int rows_groups = min(kGroups, stage_groups(G) - g0) * kRows;
    // Opaque, so that the addresses that follow from it are computed here and not
    // kept in registers through the streaming loops.
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    started();
    __builtin_amdgcn_sched_barrier(0);
    u32x4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int o = i * kThreads + tid;
        const int g = g0 + o / 8 / kRows;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (o / 8 < rows_groups && g < G)
            v[i] = load(o / 8 % kRows, g * 8 + o % 8);
    }
    __syncthreads();  // what was there has been read
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int o = i * kThreads + tid;
        if (o / 8 < rows_groups)
            put_chunk<kRows>(operands, sums, o / 8 % kRows, o / 8 / kRows * 8 + o % 8, v[i]);
    }
    __syncthreads();
}

}  // namespace ck
