// Low-rank adapters of many requests beside a shared projection:
//   out[m] = base[m] + scaling[a] B_a (A_a x_m),  a = index[m] (outside [0, L): base[m]).
//
// Two launches: v = A_a x_m (fp32, in parts of the K columns so that few rows still
// fill the chip), then base + B_a v.  Rows of one adapter share its weights: the 64
// lanes of a wave read the indices of a window of rows, a ballot gives the rows of
// one adapter (a set), and those rows, wherever they lie in the window, fill
// the 16-row tiles of the bf16 MFMA.  Few rows: a workgroup is started for every
// tile the sets of a window can have, so that requests of unlike adapters run side
// by side; many rows (prompts, where neighbours share an adapter): a workgroup
// goes through the sets of its window.
// The work is bound by memory: x, base and out once, the used adapters once; few
// rows by the two kernels' latency (one row, K = N = 3840, rank 16: 4.0 + 5.2 us).
// Measured (durations in a kernel trace): 32 rows of as many adapters, N 10240, rank 16:
// 5.2 + 6.9 us (8 MB); 301 rows of 7, K 10240, N 3840, rank 40: 13 + 8 us (16 MB); 8192
// rows of 8 in runs, K 3840, N 10240, rank 64: 37 + 112 us (63 MB of x, 336 MB of base and
// out; the waves of the second wait 61 % of their time, and it reads 227 MB from beyond
// the L2s where base, v and B are 183).
// A x goes to the second product as two bf16 (16 significant bits), because one would add as
// much error as the result's own rounding.
#include <type_traits>

#include "rows_device.h"
#include "rows_launch.h"

namespace ck {
namespace {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kRankBlock = kLoraRankBlock;  // ranks per workgroup (first product) or pass (second)

// The rows of a window that share one adapter.
struct RowSet {
    int adapter;  // -1: none
    int order;    // lane i: the i-th row of the set (window-relative)
    int count;
};

// Lane i: the adapter of the window's row i (-1: none, -2: no such row).
__device__ __forceinline__ int window_adapter(const int32_t *index, int64_t M, int64_t L, int64_t row0, int win)
{
    const int lane = threadIdx.x % kWave;
    if (lane >= win || row0 + lane >= M)
        return -2;
    const int a = index[row0 + lane];
    return a < 0 || a >= L ? -1 : a;
}
// The set of the window's first row in `left`, which it leaves.
__device__ __forceinline__ RowSet take_set(int mine, uint64_t &left)
{
    const int lane = threadIdx.x % kWave;
    RowSet r;
    r.adapter = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t mask = __ballot(mine == r.adapter), below = (uint64_t(1) << lane) - 1;
    left &= ~mask;
    r.count = __builtin_popcountll(mask);
    const int pos = (mask >> lane) & 1 ? __builtin_popcountll(mask & below)
                                       : r.count + __builtin_popcountll(~mask & below);
    r.order = __builtin_amdgcn_ds_permute(4 * pos, lane);
    return r;
}
// The sets of the rows whose adapter is at least `from`.  Few rows (kTile): calls
// f(set, first row) for the slot-th tile of 16 rows of them, if there is one.
// Many: f(set, 0) for each set.
template <bool kTile, class F>
__device__ __forceinline__ void for_sets(int mine, int from, int slot, F &&f)
{
    uint64_t left = __ballot(mine >= from);
    if constexpr (kTile) {
        while (left) {
            const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
            const uint64_t mask = __ballot(mine == a);
            const int tiles = (__builtin_popcountll(mask) + 15) / 16;
            if (slot < tiles) {
                f(take_set(mine, left), 16 * slot);
                break;
            }
            slot -= tiles;
            left &= ~mask;
        }
    } else {
        while (left)
            f(take_set(mine, left), 0);
    }
}

__device__ __forceinline__ int adapter_rank(const int32_t *ranks, int a, int R)
{
    return ranks ? min(max(ranks[a], 0), R) : R;
}

// ---------------------------------------------------------------- first product

constexpr int kRT = kRankBlock / 16;

// Sums over the waves of the 16-row, 16-rank tiles in s_red, to v.
template <int kWaves, int kTiles>
__device__ __forceinline__ void store_v(const float (&s_red)[kWaves][kTiles][kRT][256], const int *s_rows, int p0, int count,
                                        int nrt, int rb, int rank, int R, int64_t row0, float *v)
{
    for (int o = threadIdx.x; o < kTiles * nrt * 256; o += kWaves * kWave) {
        const int r = o % 16, row = o / 16 % 16, tile = o / 256, rt = tile % nrt, mt = tile / nrt;
        const int p = p0 + 16 * mt + row;
        if (p < count && rb + 16 * rt + r < rank) {
            const int at = (row % 4) * kWave + (row / 4) * 16 + r;
            float t = s_red[0][mt][rt][at];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                t += s_red[w][mt][rt][at];
            v[(row0 + s_rows[p]) * R + rb + 16 * rt + r] = t;
        }
    }
}

// Few rows.  Grid: (windows x slots, parts of K, blocks of 64 ranks); the
// workgroup's waves split its part of K.  Operands come straight to registers,
// kAhead groups at a time: these calls are bound by latency, not by the address
// path.  Rows split over parts of K, so that one row's 3840 columns are read by 32
// waves of eight workgroups.
constexpr int kFewShrinkWaves = 4;

__global__ __launch_bounds__(kFewShrinkWaves * kWave) void lora_shrink_few_kernel(
    const uint16_t *__restrict__ x, int64_t M, int K, int64_t ldx, const int32_t *__restrict__ index, int64_t L,
    int slots, int R, const uint16_t *__restrict__ a_w, const int32_t *__restrict__ ranks, float *__restrict__ v)
{
    constexpr int kAhead = 3;
    __shared__ float s_red[kFewShrinkWaves][1][kRT][256];
    __shared__ int s_rows[kWave];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, l16 = lane % 16, quarter = lane / 16;
    const int64_t row0 = (int64_t)(blockIdx.x / slots) * kLoraWindow;
    const int rb = blockIdx.z * kRankBlock;
    const int KG = K / 64, parts = gridDim.y * kFewShrinkWaves, part = blockIdx.y * kFewShrinkWaves + wave;
    const int g0 = (int)((int64_t)part * KG / parts), g1 = (int)((int64_t)(part + 1) * KG / parts);
    const int mine = window_adapter(index, M, L, row0, kLoraWindow);
    for_sets<true>(mine, 0, blockIdx.x % slots, [&](const RowSet &rows, int p0) {
        // All ranks of the slot: the loads do not wait for the adapter's own rank.
        const int rank = adapter_rank(ranks, rows.adapter, R);
        const int nrt = min(kRT, (R - rb + 15) / 16);
        const uint16_t *arow[kRT];
#pragma unroll
        for (int rt = 0; rt < kRT; ++rt)
            arow[rt] = a_w + ((int64_t)rows.adapter * R + min(rb + 16 * rt + l16, R - 1)) * K + 16 * quarter;
        const uint16_t *xrow = x + (row0 + __shfl(rows.order, min(p0 + l16, rows.count - 1))) * ldx + 16 * quarter;
        if (wave == 0)
            s_rows[lane] = rows.order;
        v4f acc[kRT];
#pragma unroll
        for (int rt = 0; rt < kRT; ++rt)
            acc[rt] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int gb = g0; gb < g1; gb += kAhead) {
            u32x4 xv[kAhead][2], av[kAhead][kRT][2];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (gb + u < g1)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        xv[u][h] = *reinterpret_cast<const u32x4 *>(xrow + (gb + u) * 64 + 8 * h);
#pragma unroll
                        for (int rt = 0; rt < kRT; ++rt)
                            if (rt < nrt)
                                av[u][rt][h] = *reinterpret_cast<const u32x4 *>(arow[rt] + (gb + u) * 64 + 8 * h);
                    }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (gb + u < g1)
#pragma unroll
                    for (int rt = 0; rt < kRT; ++rt)
                        if (rt < nrt)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                acc[rt] = mfma16(__builtin_bit_cast(v8bf, xv[u][h]),
                                                 __builtin_bit_cast(v8bf, av[u][rt][h]), acc[rt]);
        }
#pragma unroll
        for (int rt = 0; rt < kRT; ++rt)
            if (rt < nrt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s_red[wave][0][rt][i * kWave + lane] = acc[rt][i];
        __syncthreads();
        store_v<kFewShrinkWaves, 1>(s_red, s_rows, p0, rows.count, nrt, rb, rank, R, row0,
                                    v + (int64_t)blockIdx.y * M * R);
    });
}

// Many rows.  Grid: (windows, parts of K, blocks of 64 ranks).  Each wave
// streams its part of the columns of the set's rows of x and of the adapter's rows
// through an LDS ring of its own: a stage is 64 columns, every instruction eight
// rows of 128 contiguous bytes, with the 16-byte slots XORed by the row's low bits so
// that the operand reads are free of bank conflicts.  (In operand order straight
// to registers: 48 us for 8192 rows of rank 64, against 37.)
constexpr int kManyShrinkWaves = 4, kManyStages = 2, kMT = kLoraWindow / 16;
constexpr int kManyStageBytes = (kLoraWindow + kRankBlock) * 128;

// At most n instructions outstanding (n even, up to 16); they retire in order.
__device__ __forceinline__ void wait_even(int n)
{
    switch (n / 2) {
    case 2: __builtin_amdgcn_s_waitcnt(4 | 0x0F70); break;
    case 3: __builtin_amdgcn_s_waitcnt(6 | 0x0F70); break;
    case 4: __builtin_amdgcn_s_waitcnt(8 | 0x0F70); break;
    case 5: __builtin_amdgcn_s_waitcnt(10 | 0x0F70); break;
    case 6: __builtin_amdgcn_s_waitcnt(12 | 0x0F70); break;
    case 7: __builtin_amdgcn_s_waitcnt(14 | 0x0F70); break;
    case 8: __builtin_amdgcn_s_waitcnt(0x4F70); break;  // 16
    default: wait_vmcnt0(); break;
    }
}

__global__ __launch_bounds__(kManyShrinkWaves * kWave) void lora_shrink_many_kernel(
    const uint16_t *__restrict__ x, int64_t M, int K, int64_t ldx, const int32_t *__restrict__ index, int64_t L,
    int R, const uint16_t *__restrict__ a_w, const int32_t *__restrict__ ranks, float *__restrict__ v)
{
    // The rings; after the products, the waves' sums.
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[kManyShrinkWaves][kManyStages * kManyStageBytes];
    __shared__ int s_rows[kWave];
    static_assert(sizeof s_ring >= kManyShrinkWaves * kMT * kRT * 256 * 4, "sums");
    float(&s_red)[kManyShrinkWaves][kMT][kRT][256] =
        *reinterpret_cast<float(*)[kManyShrinkWaves][kMT][kRT][256]>(&s_ring);
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, l16 = lane % 16, quarter = lane / 16;
    const int64_t row0 = (int64_t)blockIdx.x * kLoraWindow;
    const int rb = blockIdx.z * kRankBlock;
    const int KG = K / 64, parts = gridDim.y * kManyShrinkWaves, part = blockIdx.y * kManyShrinkWaves + wave;
    const int g0 = (int)((int64_t)part * KG / parts), g1 = (int)((int64_t)(part + 1) * KG / parts);
    const int mine = window_adapter(index, M, L, row0, kLoraWindow);
    lds_u8 *ring = (lds_u8 *)s_ring[wave];
    const int chunk = (lane % 8) ^ (lane / 8);
    for_sets<false>(mine, 0, 0, [&](const RowSet &rows, int) {
        const int rank = adapter_rank(ranks, rows.adapter, R);
        if (rank <= rb)
            return;
        const int nrt = min(kRT, (rank - rb + 15) / 16), nmt = (rows.count + 15) / 16;
        const int each = 2 * nmt + 2 * nrt;  // instructions of a stage
        // This lane's row of each eight of x, and of the adapter.
        const uint16_t *xr[2 * kMT];
#pragma unroll
        for (int i = 0; i < 2 * kMT; ++i)
            xr[i] = x + (row0 + __shfl(rows.order, min(8 * i + lane / 8, rows.count - 1))) * ldx + 8 * chunk;
        const uint16_t *ar = a_w + ((int64_t)rows.adapter * R + rb) * K + 8 * chunk;
        const auto issue = [&](int g, int place) {
            lds_u8 *to = ring + place * kManyStageBytes;
#pragma unroll
            for (int i = 0; i < 2 * kMT; ++i)
                if (i < 2 * nmt)
                    __builtin_amdgcn_global_load_lds(
                        xr[i] + g * 64, (__attribute__((address_space(3))) void *)(to + i * 1024), 16, 0, 0);
#pragma unroll
            for (int i = 0; i < 2 * kRT; ++i)
                if (i < 2 * nrt)
                    __builtin_amdgcn_global_load_lds(
                        ar + (int64_t)min(8 * i + lane / 8, rank - rb - 1) * K + g * 64,
                        (__attribute__((address_space(3))) void *)(to + (2 * kMT + i) * 1024), 16, 0, 0);
        };
        v4f acc[kMT][kRT];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int rt = 0; rt < kRT; ++rt)
                acc[mt][rt] = v4f{0.f, 0.f, 0.f, 0.f};
        __syncthreads();  // the last set's sums have been read
        if (g0 < g1)
            issue(g0, 0);
        for (int g = g0; g < g1; ++g) {
            // The stage has landed once the newer one's instructions are all that is outstanding.
            if (g + 1 < g1) {
                issue(g + 1, (g + 1 - g0) % kManyStages);
                wait_even(each);
            } else {
                wait_vmcnt0();
            }
            __builtin_amdgcn_sched_barrier(0);
            const lds_u8 *stage = ring + (g - g0) % kManyStages * kManyStageBytes;
            const auto operand = [&](int row, int h) {
                return __builtin_bit_cast(v8bf, *(__attribute__((address_space(3))) const u32x4 *)(
                                                    stage + row * 128 + ((4 * h + quarter) ^ (row % 8)) * 16));
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v8bf av[kRT];
#pragma unroll
                for (int rt = 0; rt < kRT; ++rt)
                    if (rt < nrt)
                        av[rt] = operand(kLoraWindow + 16 * rt + l16, h);
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
                    if (mt < nmt) {
                        const v8bf xv = operand(16 * mt + l16, h);
#pragma unroll
                        for (int rt = 0; rt < kRT; ++rt)
                            if (rt < nrt)
                                acc[mt][rt] = mfma16(xv, av[rt], acc[mt][rt]);
                    }
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the stage has been read
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();  // the rings have been read
        if (wave == 0)
            s_rows[lane] = rows.order;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int rt = 0; rt < kRT; ++rt)
                if (mt < nmt && rt < nrt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s_red[wave][mt][rt][i * kWave + lane] = acc[mt][rt][i];
        __syncthreads();
        store_v<kManyShrinkWaves, kMT>(s_red, s_rows, 0, rows.count, nrt, rb, rank, R, row0,
                                       v + (int64_t)blockIdx.y * M * R);
    });
}

// --------------------------------------------------------------- second product

// The 8 ranks from r on of one row of B_a, 0 from `rank` on (whatever is stored there).
__device__ __forceinline__ u32x4 mask_ranks(u32x4 w, int r, int rank)
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q] &= (r + 2 * q < rank ? 0xffffu : 0u) | (r + 2 * q + 1 < rank ? 0xffff0000u : 0u);
    return w;
}

// Grid: windows (x slots), by columns / (64 kWaves kCols).  The workgroup brings v of a
// set's rows to LDS, scaled, as two bf16 a value (16 significant bits): per 16 ranks
// 16 first parts, then 16 second parts, the 32 columns of k of one MFMA, whose
// other operand is B_a's 16 ranks twice.  A wave then owns kCols tiles of 64 columns; the
// sums of 16 rows go through LDS so that base and out are moved in 128-byte
// runs of a row (8192 rows of rank 64: 250 us without, 132 with, in earlier forms).  Four tiles of
// base are on their way at a time (three: 123 us against 115 then); asking for the first of
// them ahead of v gains nothing (116).  Two waves a SIMD fit beside B_a's operands,
// so latency shows: 3.0 TB/s of base and out, where a copy reaches 5.4.
template <bool kSlots, int kWaves, int kCols, int kSteps, bool kWide>
__global__ __launch_bounds__(kWaves * kWave, kSlots ? 1 : 2) void lora_expand_kernel(
    const float *__restrict__ v, int parts, int64_t M, const int32_t *__restrict__ index, int64_t L, int slots, int R,
    const uint16_t *__restrict__ b_w, const float *__restrict__ scaling, const int32_t *__restrict__ ranks, int N,
    const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo)
{
    constexpr int kPitch = 64 * 4 + 16;      // sums: 16 bytes on from row to row
    constexpr int kVRows = kSlots ? 1 : 4;  // rows of v a thread has on their way
    constexpr int kAhead = kSlots || kWide ? 1 : 4;   // row tiles whose base is on its way
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ __attribute__((aligned(16))) uint8_t s_out[kWaves][16 * kPitch];
    __shared__ int s_rows[kWave];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int l16 = lane % 16, quarter = lane / 16;
    const int ctiles = (N + 64 * kWaves * kCols - 1) / (64 * kWaves * kCols);
    const int unit = blockIdx.x / ctiles;
    const int64_t row0 = (int64_t)(kSlots ? unit / slots : unit) * kLoraWindow;
    const int c0 = (blockIdx.x % ctiles * kCols * kWaves + wave) * 64;  // and every 64 kWaves on
    const int vpitch = (R + 15) / 16 * 64 + 16;  // bytes of a row of v in LDS
    int mine = window_adapter(index, M, L, row0, kLoraWindow);
    // Rows without an adapter join the window's first set, so that they cost no
    // pass of their own; their base is stored as it is.
    const uint64_t without = __ballot(mine == -1), with = __ballot(mine >= 0);
    if (with) {
        const int first = __builtin_amdgcn_readlane(mine, __builtin_ctzll(with));
        mine = mine == -1 ? first : mine;
    }

    for_sets<kSlots>(mine, -1, kSlots ? unit % slots : 0, [&](const RowSet &rows, int begin) {
        const int last = kSlots ? min(begin + 16, rows.count) : rows.count;
        const int rank = rows.adapter < 0 ? 0 : adapter_rank(ranks, rows.adapter, R);
        const float scale = rows.adapter >= 0 && scaling ? scaling[rows.adapter] : 1.f;
        // Few rows: every rank of the slot is loaded, so that no load waits for the
        // adapter's own rank; what lies beyond it meets zeros, and is masked.
        const int upto = kSlots ? (rows.adapter < 0 ? 0 : R) : rank;
        const int passes = kWide ? max(1, (upto + kRankBlock - 1) / kRankBlock) : 1;
        u32x4 bf[kSteps][4];
        const auto load_b = [&](int n0, int pass) {
            int ranks_here = upto;  // opaque, as below
            if constexpr (!kWide)
                asm volatile("" : "+s"(ranks_here));
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const int r = pass * kRankBlock + 16 * st + 8 * (quarter % 2);
                if (pass * kRankBlock + 16 * st < ranks_here)
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int n = min(n0 + 16 * h + l16, N - 1);
                        bf[st][h] = u32x4{0u, 0u, 0u, 0u};
                        if (r < ranks_here)
                            bf[st][h] = *reinterpret_cast<const u32x4 *>(
                                b_w + ((int64_t)rows.adapter * N + n) * R + r);
                    }
            }
        };
        const bool ragged = rank % 8 != 0 || rank < upto;
        const auto mask_b = [&](int pass) {
            if (!ragged)
                return;
            int end = rank;  // opaque: the masks are made here, not kept in registers
            asm volatile("" : "+s"(end));
#pragma unroll
                for (int st = 0; st < kSteps; ++st)
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        bf[st][h] = mask_ranks(bf[st][h], pass * kRankBlock + 16 * st + 8 * (quarter % 2), end);
        };
        // base of a tile: two rows a lane, lane / 8 and 8 + lane / 8.
        u32x4 bv[kAhead][2];
        const auto load_base = [&](int n0, int p0, u32x4(&to)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // Past the set or the columns: the last ones again, which are not stored.
                const int p = min(p0 + 8 * i + lane / 8, last - 1), n = min(n0 + lane % 8 * 8, N - 8);
                const int row = __shfl(rows.order, p);
                to[i] = u32x4{0u, 0u, 0u, 0u};
                if (base)
                    to[i] = *reinterpret_cast<const u32x4 *>(base + (row0 + row) * ldb + n);
            }
        };
        if (c0 < N && passes == 1)
            load_b(c0, 0);
        if (kSlots && c0 < N)
            load_base(c0, begin, bv[0]);

        if (!kSlots)
            __syncthreads();  // the last set's v has been read
        if (wave == 0)
            s_rows[lane] = rows.order | (int)(without >> rows.order & 1) << 6;
        __syncthreads();
        // v to LDS: a thread takes 4 ranks of a row, 16 threads 64.
        for (int pb = begin + threadIdx.x / 16; pb < last; pb += kWaves * 4 * kVRows) {
            for (int r = threadIdx.x % 16 * 4; r < upto; r += 64) {
                v4f t[kVRows];
                const float *from[kVRows];
#pragma unroll
                for (int i = 0; i < kVRows; ++i) {
                    t[i] = v4f{0.f, 0.f, 0.f, 0.f};
                    from[i] = v + (row0 + s_rows[min(pb + kWaves * 4 * i, last - 1)] % 64) * R + r;
                }
#pragma unroll kVRows == 1 ? 2 : 1
                for (int s = 0; s < parts; ++s)
#pragma unroll
                    for (int i = 0; i < kVRows; ++i)
                        t[i] += *reinterpret_cast<const v4f *>(from[i] + s * M * R);
#pragma unroll
                for (int i = 0; i < kVRows; ++i) {
                    __builtin_amdgcn_sched_barrier(0);  // one row's masks at a time
                    const int p = pb + kWaves * 4 * i;
                    if (p >= last)
                        break;
                    const int end = s_rows[p] < 64 ? rank : 0;  // v is written up to there
                    uint16_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        split_bf16(r + e < end ? scale * t[i][e] : 0.f, hi[e], lo[e]);
                    uint8_t *to = smem + (p - begin) * vpitch + r / 16 * 64 + r % 16 * 2;
                    *reinterpret_cast<u32x2 *>(to) = u32x2{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16};
                    *reinterpret_cast<u32x2 *>(to + 32) =
                        u32x2{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16};
                }
            }
        }
        for (int p = begin + threadIdx.x / 16; p < last; p += kWaves * 4) {
            // The other half of the last 16 ranks.
            const int end = (upto + 3) / 4 * 4;
            for (int r = end + threadIdx.x % 16 * 4; r % 16 != 0 && r < (end + 15) / 16 * 16; r += 64) {
                uint8_t *to = smem + (p - begin) * vpitch + r / 16 * 64 + r % 16 * 2;
                *reinterpret_cast<u32x2 *>(to) = *reinterpret_cast<u32x2 *>(to + 32) = u32x2{0u, 0u};
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int ct = 0; ct < kCols; ++ct) {
            const int n0 = c0 + 64 * kWaves * ct, n = n0 + lane % 8 * 8;
            if (n0 >= N)
                break;
            if (passes == 1) {
                if (ct > 0)
                    load_b(n0, 0);
                mask_b(0);
            }
            for (int pb = begin; pb < last; pb += 16 * kAhead) {
                if (!kSlots || ct > 0)
#pragma unroll
                    for (int i = 0; i < kAhead; ++i)
                        load_base(n0, pb + 16 * i, bv[i]);
#pragma unroll
                for (int tile = 0; tile < kAhead; ++tile) {
                    const int p0 = pb + 16 * tile;
                    if (p0 >= last)
                        break;
                    __builtin_amdgcn_sched_barrier(0);
                    int ranks_here = upto;  // opaque: compared here, not once for all tiles
                    if constexpr (!kWide)
                        asm volatile("" : "+s"(ranks_here));
                    v4f acc[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        acc[h] = v4f{0.f, 0.f, 0.f, 0.f};
                    for (int pass = 0; pass < passes; ++pass) {
                        if (passes > 1) {
                            load_b(n0, pass);
                            mask_b(pass);
                        }
#pragma unroll
                        for (int st = 0; st < kSteps; ++st) {
                            const int r = pass * kRankBlock + 16 * st;
                            if (r < ranks_here) {
                                // Rows past the set repeat its last one and are not stored.
                                const v8bf vf = *reinterpret_cast<const v8bf *>(
                                    smem + (min(p0 + l16, last - 1) - begin) * vpitch + r * 4 + quarter * 16);
#pragma unroll
                                for (int h = 0; h < 4; ++h)
                                    acc[h] = mfma16(__builtin_bit_cast(v8bf, bf[st][h]), vf, acc[h]);
                            }
                        }
                    }
                    // Lane l16 is the row, registers i the columns 16 h + 4 quarter + i.
                    uint8_t *sums = s_out[wave];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        *reinterpret_cast<v4f *>(sums + l16 * kPitch + (16 * h + 4 * quarter) * 4) = acc[h];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int p = p0 + 8 * i + lane / 8;
                        const uint8_t *from = sums + (8 * i + lane / 8) * kPitch + lane % 8 * 32;
                        const v4f t0 = *reinterpret_cast<const v4f *>(from), t1 = *reinterpret_cast<const v4f *>(from + 16);
                        if (p < last && n < N) {
                            const int row = s_rows[p];
                            const u32x4 y = bv[tile][i];
                            u32x4 o;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const v4f &t = q < 2 ? t0 : t1;
                                o[q] = pack_bf16x2(t[2 * q % 4] + bf16_to_f32(y[q] & 0xffffu),
                                                   t[2 * q % 4 + 1] + __uint_as_float(y[q] & 0xffff0000u));
                                o[q] = row < 64 ? o[q] : y[q];
                            }
                            *reinterpret_cast<u32x4 *>(out + (row0 + row % 64) * ldo + n) = o;
                        }
                    }
                }
            }
        }
    });
}

struct ExpandArgs {
    const float *v;
    int parts;
    int64_t M;
    const int32_t *index;
    int64_t L;
    int slots, R;
    const uint16_t *b;
    const float *scaling;
    const int32_t *ranks;
    int N;
    const uint16_t *base;
    int64_t ldb;
    uint16_t *out;
    int64_t ldo;
};

template <bool kSlots, int kWaves, int kCols, int kSteps, bool kWide = false>
hipError_t launch_expand(const ExpandArgs &a, hipStream_t s)
{
    const auto kernel = lora_expand_kernel<kSlots, kWaves, kCols, kSteps, kWide>;
    const int lds = (kSlots ? 16 : kLoraWindow) * ((a.R + 15) / 16 * 64 + 16);  // at most 65 KiB
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, 72 * 1024);
    if (attr != hipSuccess)
        return attr;
    const int64_t blocks =
        lora_ceil(a.M, kLoraWindow) * (kSlots ? a.slots : 1) * lora_ceil(a.N, 64 * kWaves * kCols);
    if (blocks * kWaves * kWave >= int64_t(1) << 32)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kWaves * kWave), lds, s, a.v, a.parts, a.M, a.index, a.L,
                       a.slots, a.R, a.b, a.scaling, a.ranks, a.N, a.base, a.ldb, a.out, a.ldo);
    return hipGetLastError();
}

template <bool kSlots, int kWaves, int kCols>
hipError_t launch_expand_steps(const ExpandArgs &a, hipStream_t s)
{
    // As many of B_a's operands in registers as R needs: fewer leave room for more
    // waves.  Beyond 64 ranks they are loaded for every row tile, 64 ranks at a time.
    return a.R <= 16   ? launch_expand<kSlots, kWaves, kCols, 1>(a, s)
           : a.R <= 32 ? launch_expand<kSlots, kWaves, kCols, 2>(a, s)
           : a.R <= kRankBlock ? launch_expand<kSlots, kWaves, kCols, 4>(a, s)
                               : launch_expand<kSlots, kWaves, kCols, 4, true>(a, s);
}

}  // namespace

int launch_lora(const uint16_t *x, int64_t M, int K, int64_t ldx, const int32_t *index, int64_t L, int R,
                const uint16_t *a, const uint16_t *b, const float *scaling, const int32_t *ranks, int N,
                const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo, float *ws, void *stream)
{
    if (M <= 0)
        return 0;
    if (K % 64 != 0 || R % 8 != 0 || R < 8 || R > kLoraMaxRank || N % 16 != 0 || L < 1)
        return (int)hipErrorInvalidValue;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int parts = lora_splits(M, K, R, L), slots = lora_slots(M, L);
    const int64_t windows = lora_ceil(M, kLoraWindow);
    const bool few = M <= kLoraFewRows;
    const dim3 grid((unsigned)(windows * (few ? slots : 1)), parts, (unsigned)lora_ceil(R, kRankBlock));
    if (few)
        hipLaunchKernelGGL(lora_shrink_few_kernel, grid, dim3(kFewShrinkWaves * kWave), 0, s, x, M, K, ldx, index, L,
                           slots, R, a, ranks, ws);
    else
        hipLaunchKernelGGL(lora_shrink_many_kernel, grid, dim3(kManyShrinkWaves * kWave), 0, s, x, M, K, ldx, index, L,
                           R, a, ranks, ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return (int)e;
    const ExpandArgs ea{ws, parts, M, index, L, slots, R, b, scaling, ranks, N, base, ldb, out, ldo};
    if (!few)
        e = launch_expand_steps<false, 4, 2>(ea, s);
    else if (lora_expand_waves(M, L, R, N) == 1)
        e = launch_expand_steps<true, 1, 1>(ea, s);
    else
        e = launch_expand_steps<true, 4, 1>(ea, s);
    return (int)e;
}

}  // namespace ck
