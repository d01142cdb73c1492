// Mixture-of-experts layer on packed uint4 experts (AWQ W4A16) for few tokens.
//
//   W[n, c] = (q - 8) s[c / 64, n] + z[c / 64, n], kept exact,
//   h = silu(W1[e][:I] x) * (W1[e][I:] x),  y = W2[e] h,
//   out[t] = sum over the token's slots j of weight_j y_{e_j}.
//
// Few tokens make this a matter of streaming the chosen experts' weights once
// (w4_stream.h), whatever the number of tokens each has.  Sums are fp32; h goes
// to the second product as two bf16 (16 significant bits), as two rows of A.
//
// Launches, for P = tokens * k (token, slot) pairs:
//   few pairs:  first product (each workgroup routes its token itself), second
//               product with the weighted sum: two launches;
//   otherwise:  router, first product, second product, weighted sum.  Each
//               workgroup collects its expert's pairs from the ids with ballots.
#include "moe_route.h"
#include "rows_launch.h"
#include "w4_stream.h"

namespace ck {
namespace {

// ---------------------------------------------------------------- first product

struct UpArgs {
    const uint16_t *x;
    int64_t ldx;
    int k;
    const uint8_t *w1;
    const uint16_t *s1, *z1;
    int E, H, I, P;
    MoeRouting r;
    uint16_t *hidden;         // [P][2][I]: first parts, second parts
};

// silu(g) u of hidden column n of a pair, as two bf16.
__device__ __forceinline__ void put_hidden(uint16_t *hidden, int pair, int I, int n, float g, float u)
{
    uint16_t hi, lo;
    split_bf16(g / (1.f + expf(-g)) * u, hi, lo);
    uint16_t *dst = hidden + (int64_t)pair * 2 * I + n;
    dst[0] = hi;
    dst[I] = lo;
}

constexpr int kFewUpWaves = 4;

// Few pairs.  A unit is a pair, routed here (kNe logits a lane) or by the given
// ids (kNe 0); a workgroup owns 16 hidden columns of it, a wave's tile being
// their 16 gate and 16 up rows, and the waves split the H columns.
template <int kNe, bool kBf16>
__global__ __launch_bounds__(kFewUpWaves * kWave) void moe_up_few_kernel(const UpArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // rings, operands, sums
    __shared__ float s_red[kFewUpWaves][32];
    const int H = p.H, I = p.I, G = H / 64, tiles = I / 16;
    // Neighbouring tiles share lines of the scales: runs of four go to one XCD.
    const int local = blockIdx.x / kXcds, run = local / 4 * kXcds + blockIdx.x % kXcds;
    const int y = run / (tiles / 4), n0 = (run % (tiles / 4) * 4 + local % 4) * 16;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, l32 = lane % 32;
    if (y >= p.P)
        return;
    const int t = y / p.k, slot = y - t * p.k;
    int e;
    if constexpr (kNe > 0) {
        int id;
        float wt;
        route_row<kNe, kBf16>(static_cast<const uint8_t *>(p.r.logits) + (int64_t)t * p.r.ldl * (kBf16 ? 2 : 4), p.E,
                              p.k, p.r.renormalize, lane, id, wt);
        if (slot == 0 && n0 == 0 && threadIdx.x < p.k) {
            p.r.ids[t * p.k + lane] = id;
            p.r.weights[t * p.k + lane] = wt;
        }
        e = __builtin_amdgcn_readlane(id, slot);
    } else {
        e = __builtin_amdgcn_readfirstlane(p.r.ids[y]);
    }
    if (e < 0 || e >= p.E)
        return;
    const int stages = (G + kStageGroups - 1) / kStageGroups;
    const int st0 = wave * stages / kFewUpWaves, st1 = (wave + 1) * stages / kFewUpWaves;
    WeightStream ws(p.w1, p.s1, p.z1, 2 * I, G, I, smem + wave * kRingBytes);
    OneTile cursor{st0, st1};
    ws.tile(e, n0);
    ws.start(cursor);
    uint8_t *operands = smem + kFewUpWaves * kRingBytes;
    const int GP = stage_groups(G);
    float *sums = reinterpret_cast<float *>(operands + GP * 128);
    const uint16_t *x = p.x + (int64_t)t * p.ldx;
    for (int c = threadIdx.x; c < GP * 8; c += kFewUpWaves * kWave) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (c < G * 8)
            v = __builtin_bit_cast(u32x4, act_order8(*reinterpret_cast<const u32x4 *>(x + c * 8)));
        put_chunk<1>(operands, sums, 0, c, v);
    }
    __syncthreads();
    float tot[1] = {0.f};
    stream_stages<1>(ws, cursor, p.z1 != nullptr, st0, st1, 0, ARows<1>{operands, sums}, tot, [] {});
    if (lane < 32)
        s_red[wave][l32] = tot[0];
    __syncthreads();
    if (threadIdx.x < 16) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kFewUpWaves; ++w)
            g += s_red[w][l32], u += s_red[w][l32 + 16];
        put_hidden(p.hidden, y, I, n0 + l32, g, u);
    }
}

// ------------------------------------------------------------- many pairs: work
//
// An expert's pairs are taken in sets of up to eight (a second set reads the
// weights again), and a set's 32-row weight tiles in octets, a tile for each wave.
// One workgroup fits a CU, and each takes an equal run of the octets of all
// sets, so that no CU ends late because an expert has many pairs or because
// the chosen experts do not divide the chip.  A workgroup finds its run from the
// ids itself; a wave's weights are one stream through all its tiles.
constexpr int kWaves = 8, kSetPairs = 8, kMaxSets = 8;

struct Shared {
    uint8_t ring[kWaves][kRingBytes];
    uint8_t operands[kChunkOperands];
    float sums[kChunkSums];
    int expert[kMaxSets], count[kMaxSets];
    uint16_t pairs[kMaxSets][kSetPairs];
};
static_assert(sizeof(int) * kRouteMaxExperts <= kChunkOperands, "the experts' counts lie in the operands' place");

struct Run {
    int q0, q1;      // octets, counted through all sets
    int first_set;   // its sets are in Shared from here on
};

__device__ __forceinline__ int wave_sum_int(int v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ Run plan_run(const int32_t *ids, int P, int E, int octets, Shared &s)
{
    int *cnt = reinterpret_cast<int *>(s.operands);
    const int t = threadIdx.x, lane = t % kWave, wave = t / kWave;
    for (int e = t; e < E; e += kWaves * kWave)
        cnt[e] = 0;
    __syncthreads();
    for (int p = t; p < P; p += kWaves * kWave) {
        const int e = ids[p];
        if (e >= 0 && e < E)
            atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    int sets = 0;
    for (int c = 0; c < E; c += kWave)
        sets += c + lane < E ? (cnt[c + lane] + kSetPairs - 1) / kSetPairs : 0;
    sets = wave_sum_int(sets);
    const int total = sets * octets;
    Run r;
    r.q0 = (int)((int64_t)total * blockIdx.x / gridDim.x);
    r.q1 = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    r.first_set = r.q0 / octets;
    // Wave i finds the run's i-th set: its expert, and its pairs in ascending order.
    const int set = r.first_set + wave;
    if (r.q0 < r.q1 && set <= (r.q1 - 1) / octets) {
        int before = 0, expert = 0, first = 0, count = 0;
        for (int c = 0; c < E; c += kWave) {
            const int n = c + lane < E ? cnt[c + lane] : 0;
            int v = (n + kSetPairs - 1) / kSetPairs;
            const int own = v;
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) {
                const int u = __shfl_up(v, d);
                if (lane >= d)
                    v += u;
            }
            const uint64_t here = __ballot(before + v - own <= set && set < before + v);
            if (here) {
                const int l = __builtin_ctzll(here);
                expert = c + l;
                first = (set - before - __builtin_amdgcn_readlane(v - own, l)) * kSetPairs;
                count = __builtin_amdgcn_readlane(n, l) - first;
                break;
            }
            before += __builtin_amdgcn_readlane(v, kWave - 1);
        }
        int seen = -first;
        for (int c = 0; c < P && seen < kSetPairs; c += kWave) {
            const uint64_t mask = __ballot(c + lane < P && ids[c + lane] == expert);
            const int at = seen + __builtin_popcountll(mask & ((uint64_t(1) << lane) - 1));
            if ((mask >> lane & 1) && at >= 0 && at < kSetPairs)
                s.pairs[wave][at] = (uint16_t)(c + lane);
            seen += __builtin_popcountll(mask);
        }
        if (lane == 0)
            s.expert[wave] = expert, s.count[wave] = min(count, kSetPairs);
    }
    __syncthreads();
    return r;
}

// Cursor over a wave's tiles of a run: tile `wave` of each octet, where there is one.
struct RunCursor {
    const int *expert;
    int q, q1, first_set, octets, tiles, rows, wave, st, stages;
    __device__ __forceinline__ RunCursor(const Run &r, const Shared &s, int octets_, int tiles_, int rows_, int stages_)
        : expert(s.expert), q(r.q0), q1(r.q1), first_set(r.first_set), octets(octets_), tiles(tiles_), rows(rows_),
          wave(threadIdx.x / kWave), st(0), stages(stages_)
    {
    }
    __device__ __forceinline__ bool next(WeightStream &ws, int &stage)
    {
        if (st == 0) {
            while (q < q1 && q % octets * kWaves + wave >= tiles)
                ++q;
            if (q >= q1)
                return false;
            ws.tile(__builtin_amdgcn_readfirstlane(expert[q / octets - first_set]),
                    (q % octets * kWaves + wave) * rows);
        }
        stage = st;
        if (++st == stages)
            st = 0, ++q;
        return true;
    }
};

// Octets [q0, q1) of one set against kRows rows of A.  done(tile, tot).
template <int kRows, class Load, class Done>
__device__ __forceinline__ void stream_set(WeightStream &ws, RunCursor &cursor, bool zeros, int q0, int q1, bool start,
                                           Shared &s, Load &&load, Done &&done)
{
    constexpr int kGroups = kChunkElems / 64 / kRows, kRegs = ARows<kRows>::kRegs;
    const int G = ws.G, stages = cursor.stages, wave = threadIdx.x / kWave;
    const ARows<kRows> A{s.operands, s.sums};
    const bool whole = G <= kGroups;
    float tot[kRegs], held[kRegs];
    int held_tile = -1;
    const auto flush = [&] {
        if (held_tile >= 0)
            done(held_tile, held);
        held_tile = -1;
    };
    for (int q = q0; q < q1; ++q) {
        const int tile = q % cursor.octets * kWaves + wave;
#pragma unroll
        for (int i = 0; i < kRegs; ++i)
            tot[i] = 0.f;
        for (int g0 = 0; g0 < G; g0 += kGroups) {
            if (!whole || q == q0)
                fill_rows<kRows, kWaves>(G, g0, s.operands, s.sums, load, [&] {
                    if (start && q == q0 && g0 == 0)
                        ws.start(cursor);
                });
            if (tile < cursor.tiles)
                stream_stages<kRows>(ws, cursor, zeros, g0 / kStageGroups,
                                     min(stages, (g0 + kGroups) / kStageGroups), g0, A, tot, flush);
        }
        if (tile < cursor.tiles) {
            held_tile = tile;
#pragma unroll
            for (int i = 0; i < kRegs; ++i)
                held[i] = tot[i];
        }
    }
    flush();
}

// The first product of many pairs: a tile is 16 hidden columns (their gate and up
// rows); A's rows are the set's tokens.
template <int kRows>
__device__ __forceinline__ void up_set(const UpArgs &p, WeightStream &ws, RunCursor &cursor, int set, int q0, int q1,
                                       bool start, Shared &s)
{
    const int lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32, count = s.count[set];
    const auto load = [&](int row, int ch) {
        const int pr = s.pairs[set][min(row, count - 1)];
        return __builtin_bit_cast(
            u32x4, act_order8(*reinterpret_cast<const u32x4 *>(p.x + (int64_t)(pr / p.k) * p.ldx + ch * 8)));
    };
    const auto done = [&](int tile, const float(&tot)[ARows<kRows>::kRegs]) {
#pragma unroll
        for (int i = 0; i < ARows<kRows>::kRegs; ++i) {
            const float u = __shfl_xor(tot[i], 16);
            const int row = (kRows > 4 ? 4 * half : 0) + i;
            if (l32 < 16 && (kRows > 4 || half == 0) && row < count)
                put_hidden(p.hidden, s.pairs[set][row], p.I, tile * 16 + l32, tot[i], u);
        }
    };
    stream_set<kRows>(ws, cursor, p.z1 != nullptr, q0, q1, start, s, load, done);
}

__global__ __launch_bounds__(kWaves * kWave, 2) void moe_up_kernel(const UpArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int tiles = p.I / 16, octets = (tiles + kWaves - 1) / kWaves, G = p.H / 64;
    const Run r = plan_run(p.r.ids, p.P, p.E, octets, s);
    WeightStream ws(p.w1, p.s1, p.z1, 2 * p.I, G, p.I, s.ring[threadIdx.x / kWave]);
    RunCursor cursor(r, s, octets, tiles, 16, stage_groups(G) / kStageGroups);
    for (int q = r.q0; q < r.q1;) {
        const int set = q / octets - r.first_set, end = min(r.q1, (q / octets + 1) * octets);
        if (s.count[set] <= 4)
            up_set<4>(p, ws, cursor, set, q, end, q == r.q0, s);
        else
            up_set<8>(p, ws, cursor, set, q, end, q == r.q0, s);
        q = end;
    }
}

// --------------------------------------------------------------- second product

struct DownArgs {
    const uint16_t *hidden;
    const uint8_t *w2;
    const uint16_t *s2, *z2;
    int E, H, I, T, k;
    const int32_t *ids;
    const float *weights;
    float *y;                 // [P][H]
    uint16_t *out;
    int64_t ldo;
};

constexpr int kFewWaves = 8;

// Few pairs: a workgroup owns 32 output columns; its waves take the pairs (or
// slices of the I columns, where there are fewer pairs than waves), then every
// output adds its token's slots in order.  A has a pair's first parts in its even
// rows' place and the second parts in the odd (rows 0 and 4 of the result: the
// two halves of the wave).
__global__ __launch_bounds__(kFewWaves * kWave) void moe_down_few_kernel(const DownArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // rings, operands, group sums, results
    const int H = p.H, I = p.I, G = I / 64, P = p.T * p.k;
    const int n0 = xcd_block(blockIdx.x, gridDim.x) * 32;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int l32 = lane % 32, half = lane / 32;
    const int stages = (G + kStageGroups - 1) / kStageGroups;
    const int slices = max(1, min(kFewWaves / P, stages));
    const int GP = stage_groups(G);
    uint8_t *operands = smem + kFewWaves * kRingBytes;                      // [P][2][64 GP]
    float *sums = reinterpret_cast<float *>(operands + P * GP * 256);       // [P][2][GP]
    float *s_sum = sums + 2 * P * GP;                                       // [slices][P][32]

    for (int c = threadIdx.x; c < 2 * P * GP * 8; c += kFewWaves * kWave) {
        const int row = c / (GP * 8), ch = c % (GP * 8);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (ch < G * 8)
            v = __builtin_bit_cast(
                u32x4, act_order8(*reinterpret_cast<const u32x4 *>(p.hidden + (int64_t)row * I + ch * 8)));
        put_chunk<1>(operands, sums, 0, c, v);
    }
    __syncthreads();
    for (int it = wave; it < P * slices; it += kFewWaves) {
        const int pr = it / slices, sl = it % slices;
        const int e = __builtin_amdgcn_readfirstlane(p.ids[pr]);
        if (e < 0 || e >= p.E)
            continue;
        const int st0 = sl * stages / slices, st1 = (sl + 1) * stages / slices;
        WeightStream ws(p.w2, p.s2, p.z2, H, G, 16, smem + wave * kRingBytes);
        OneTile cursor{st0, st1};
        ws.tile(e, n0);
        ws.start(cursor);  // the ring's last stage has been read into registers
        float tot[1] = {0.f};
        const ARows<1> A{operands + (2 * pr + l32 / 4 % 2) * GP * 128, sums + (2 * pr + half) * GP};
        stream_stages<1>(ws, cursor, p.z2 != nullptr, st0, st1, 0, A, tot, [] {});
        const float v = tot[0] + __shfl_xor(tot[0], 32);
        if (half == 0)
            s_sum[(sl * P + pr) * 32 + l32] = v;
    }
    __syncthreads();
    for (int o = threadIdx.x; o < p.T * 32; o += kFewWaves * kWave) {
        const int t = o / 32, col = o % 32;
        float y = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const int pr = t * p.k + j, e = p.ids[pr];
            if (e >= 0 && e < p.E) {
                float v = s_sum[pr * 32 + col];
                for (int sl = 1; sl < slices; ++sl)
                    v += s_sum[(sl * P + pr) * 32 + col];
                y = __builtin_fmaf(p.weights[pr], v, y);
            }
        }
        p.out[(int64_t)t * p.ldo + n0 + col] = f32_to_bf16(y);
    }
}

// The second product of many pairs: a tile is 32 output columns, A's rows are the
// first parts of the set's pairs, then the second parts; the sums of each pair go
// to moe_combine_kernel.
template <int kPairs>
__device__ __forceinline__ void down_set(const DownArgs &p, WeightStream &ws, RunCursor &cursor, int set, int q0,
                                         int q1, bool start, Shared &s)
{
    constexpr int kRows = 2 * kPairs, kRegs = ARows<kRows>::kRegs;
    const int lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32, count = s.count[set];
    const auto load = [&](int row, int ch) {
        const int pr = s.pairs[set][min(row % kPairs, count - 1)];
        return __builtin_bit_cast(u32x4, act_order8(*reinterpret_cast<const u32x4 *>(
                                             p.hidden + ((int64_t)pr * 2 + row / kPairs) * p.I + ch * 8)));
    };
    const auto done = [&](int tile, const float(&tot)[kRegs]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // The second parts are in the other half of the wave (4 pairs) or the other four registers (8).
            const float v = kPairs == 4 ? tot[i] + __shfl_xor(tot[i], 32) : tot[i] + tot[kRegs - 4 + i];
            const int at = kPairs == 4 ? i : 4 * half + i;
            if (at < count && (kPairs > 4 || half == i / 2))
                p.y[(int64_t)s.pairs[set][at] * p.H + tile * 32 + l32] = v;
        }
    };
    stream_set<kRows>(ws, cursor, p.z2 != nullptr, q0, q1, start, s, load, done);
}

__global__ __launch_bounds__(kWaves * kWave, 2) void moe_down_kernel(const DownArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int tiles = p.H / 32, octets = (tiles + kWaves - 1) / kWaves, G = p.I / 64;
    const Run r = plan_run(p.ids, p.T * p.k, p.E, octets, s);
    WeightStream ws(p.w2, p.s2, p.z2, p.H, G, 16, s.ring[threadIdx.x / kWave]);
    RunCursor cursor(r, s, octets, tiles, 32, stage_groups(G) / kStageGroups);
    for (int q = r.q0; q < r.q1;) {
        const int set = q / octets - r.first_set, end = min(r.q1, (q / octets + 1) * octets);
        if (s.count[set] <= 4)
            down_set<4>(p, ws, cursor, set, q, end, q == r.q0, s);
        else
            down_set<8>(p, ws, cursor, set, q, end, q == r.q0, s);
        q = end;
    }
}

// out[t] = sum over the slots, in order; four columns a thread.
__global__ __launch_bounds__(256) void moe_combine_kernel(const DownArgs p)
{
    const int per = p.H / 4;
    const int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (o >= (int64_t)p.T * per)
        return;
    const int t = (int)(o / per), n = (int)(o % per) * 4;
    v4f y = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.k; ++j) {
        const int pr = t * p.k + j, e = p.ids[pr];
        if (e >= 0 && e < p.E) {
            const v4f v = *reinterpret_cast<const v4f *>(p.y + (int64_t)pr * p.H + n);
            const float w = p.weights[pr];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = __builtin_fmaf(w, v[i], y[i]);
        }
    }
    *reinterpret_cast<u32x2 *>(p.out + (int64_t)t * p.ldo + n) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

// More than 64 KiB of dynamic LDS needs the kernel's attribute raised once.
constexpr int kMaxLds = 150 * 1024, kCus = 256;
template <auto kernel>
hipError_t allow_lds()
{
    static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds);
    return e;
}

template <int kNe, bool kBf16>
hipError_t launch_up_few(const UpArgs &a, hipStream_t s)
{
    constexpr auto kernel = moe_up_few_kernel<kNe, kBf16>;
    const hipError_t e = allow_lds<kernel>();
    if (e != hipSuccess)
        return e;
    const int runs = a.P * (a.I / 64);  // of four workgroups, rounded up to whole rounds of the XCDs
    const int lds = kFewUpWaves * kRingBytes + stage_groups(a.H / 64) * (128 + 4);
    hipLaunchKernelGGL(kernel, dim3((runs + kXcds - 1) / kXcds * kXcds * 4), dim3(kFewUpWaves * kWave), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_up(const UpArgs &a, bool few, int blocks, hipStream_t s)
{
    if (!few) {
        const hipError_t e = allow_lds<moe_up_kernel>();
        if (e != hipSuccess)
            return e;
        hipLaunchKernelGGL(moe_up_kernel, dim3(blocks), dim3(kWaves * kWave), sizeof(Shared), s, a);
        return hipGetLastError();
    }
    if (!a.r.logits)
        return launch_up_few<0, false>(a, s);
    if (a.E <= 256)
        return a.r.bf16 ? launch_up_few<4, true>(a, s) : launch_up_few<4, false>(a, s);
    return a.r.bf16 ? launch_up_few<16, true>(a, s) : launch_up_few<16, false>(a, s);
}

}  // namespace

int launch_moe(const uint16_t *x, int T, int64_t ldx, const MoeRouting &r, const MoeExperts &w, uint16_t *out,
               int64_t ldo, void *ws, void *stream)
{
    const int P = T * r.k;
    if (T < 1 || r.k < 1 || r.k > kRouteMaxK || P > kMoePairs || w.E < 1 || w.E > kRouteMaxExperts || w.H % 64 != 0 ||
        w.I % 64 != 0)
        return (int)hipErrorInvalidValue;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    uint16_t *hidden = static_cast<uint16_t *>(ws);
    float *y = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + moe_hidden_bytes(P, w.I));

    const int few_lds = kFewWaves * kRingBytes + 2 * P * stage_groups(w.I / 64) * (128 + 4) +
                        (P > kFewWaves ? P : kFewWaves) * 32 * 4;
    const bool few = P <= kMoeFewPairs && few_lds <= kMaxLds;
    if (r.logits && !few) {
        const int e = launch_moe_route(r.logits, r.bf16, T, w.E, r.ldl, r.k, r.renormalize, r.ids, r.weights, stream);
        if (e != 0)
            return e;
    }
    const UpArgs ua{x, ldx, r.k, w.w1, w.s1, w.z1, w.E, w.H, w.I, P, r, hidden};
    // One workgroup a CU, and no more than there can be octets; at most kMaxSets
    // sets a workgroup, which 256 workgroups keep to by far (up to 1152 sets).
    const int most_sets = (w.E < P ? w.E : P) + P / kSetPairs;
    const auto grid = [&](int tiles) {
        const int64_t octets = (int64_t)most_sets * ((tiles + kWaves - 1) / kWaves);
        return octets < kCus ? (int)octets : kCus;
    };
    hipError_t e = launch_up(ua, few, grid(w.I / 16), s);
    if (e != hipSuccess)
        return (int)e;
    const DownArgs da{hidden, w.w2, w.s2, w.z2, w.E, w.H, w.I, T, r.k, r.ids, r.weights, y, out, ldo};
    if (few) {
        e = allow_lds<moe_down_few_kernel>();
        if (e != hipSuccess)
            return (int)e;
        hipLaunchKernelGGL(moe_down_few_kernel, dim3(w.H / 32), dim3(kFewWaves * kWave), few_lds, s, da);
    } else {
        e = allow_lds<moe_down_kernel>();
        if (e != hipSuccess)
            return (int)e;
        hipLaunchKernelGGL(moe_down_kernel, dim3(grid(w.H / 32)), dim3(kWaves * kWave), sizeof(Shared), s, da);
        const int64_t quads = (int64_t)T * (w.H / 4);
        hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s, da);
    }
    return (int)hipGetLastError();
}

}  // namespace ck
