// Mixture-of-experts layer on packed uint4 experts (AWQ W4A16) for few tokens.
//
//   W[n, c] = (q - 8) s[c / 64, n] + z[c / 64, n], kept exact,
//   h = silu(W1[e][:I] x) * (W1[e][I:] x),  y = W2[e] h,
//   out[t] = sum over the token's slots j of weight_j y_{e_j}.
//
// Few tokens make this a matter of streaming the chosen experts' weights once
// (w4_stream.h), whatever the number of tokens each has.  Sums are fp32; h goes
// to the second product as two bf16 (16 significant bits), as two rows of A: one bf16
// would add as much error as the result's own rounding, and a third part (24 bits) a
// third row of A for what lies 2^8 below that rounding.
//
// Launches, for P = tokens * k (token, slot) pairs:
//   few pairs:  first product (each workgroup routes its token itself), second
//               product with the weighted sum: two launches;
//   otherwise:  router, first product, second product, weighted sum.  Each
//               workgroup collects its expert's pairs from the ids with ballots.
//
// Measured (H 3840, I 1280, zero points, cold weights), of about 6.1 TB/s that bare
// reads reach here; a call, and its products' durations in a kernel trace, which keeps
// the kernels of a call apart (their sum is up to a tenth more than the call): one token
// of 8 experts 25 us (first product 44 MB in 14 us, second 22 MB in 12); 64 tokens of 8
// in 128 experts 232-251 us (697 MB in 161-168, 348 MB in 91-97); 8 tokens in 64 experts,
// no zero points, 96 us (219 MB in 58, 110 MB in 35).  1.00 to 1.05 times those bytes
// come from beyond the L2s; the waves wait 37 to 48 % of their time.
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
    __shared__ int s_expert;
    const int H = p.H, I = p.I, G = H / 64, tiles = I / 16;
    // Neighbouring tiles share lines of the scales: runs of four go to one XCD.
    const int local = blockIdx.x / kXcds, run = local / 4 * kXcds + blockIdx.x % kXcds;
    const int y = run / (tiles / 4), n0 = (run % (tiles / 4) * 4 + local % 4) * 16;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, l32 = lane % 32;
    if (y >= p.P)
        return;
    const int t = y / p.k, slot = y - t * p.k;
    const int GP = stage_groups(G);
    uint8_t *operands = smem + kFewUpWaves * kRingBytes;
    float *sums = reinterpret_cast<float *>(operands + GP * 128);
    // One wave routes, as far as this slot, the others bring x to LDS meanwhile; one
    // workgroup of the token chooses every slot and writes them.
    const bool writes = slot == 0 && n0 == 0;
    int e = 0;
    Routed<(kNe > 0) ? kNe : 1> routed;
    if (kNe == 0 || wave == 0) {
        if constexpr (kNe > 0) {
            routed = route_select<kNe, kBf16>(
                static_cast<const uint8_t *>(p.r.logits) + (int64_t)t * p.r.ldl * (kBf16 ? 2 : 4), p.E,
                writes ? p.k : slot + 1, lane);
            if (lane == slot)
                s_expert = routed.id;
        } else {
            e = __builtin_amdgcn_readfirstlane(p.r.ids[y]);
        }
    }
    constexpr int kFirst = kNe > 0 ? 1 : 0;  // first wave that stages x
    if (wave >= kFirst) {
        const uint16_t *x = p.x + (int64_t)t * p.ldx;
        constexpr int kStride = (kFewUpWaves - kFirst) * kWave, kLoads = 4;
        for (int c0 = threadIdx.x - kFirst * kWave; c0 < GP * 8; c0 += kLoads * kStride) {
            u32x4 v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                v[i] = u32x4{0u, 0u, 0u, 0u};
                if (c0 + i * kStride < G * 8)
                    v[i] = __builtin_bit_cast(
                        u32x4, act_order8(*reinterpret_cast<const u32x4 *>(x + (c0 + i * kStride) * 8)));
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (c0 + i * kStride < GP * 8)
                    put_chunk<1>(operands, sums, 0, c0 + i * kStride, v[i]);
        }
    }
    __syncthreads();
    if constexpr (kNe > 0) {
        e = __builtin_amdgcn_readfirstlane(s_expert);
        if (writes && wave == 0) {
            const float wt = route_weight(routed, p.r.renormalize);
            if (lane < p.k) {
                p.r.ids[t * p.k + lane] = routed.id;
                p.r.weights[t * p.k + lane] = wt;
            }
        }
    }
    if (e < 0 || e >= p.E)
        return;
    WeightStream<> ws(p.w1, p.s1, p.z1, 2 * I, G, I, smem + wave * kRingBytes);
    const int stages = ws.stages();
    const int st0 = wave * stages / kFewUpWaves, st1 = (wave + 1) * stages / kFewUpWaves;
    OneTile cursor{st0, st1};
    ws.tile(e, n0);
    ws.start(cursor);
    float tot[1] = {0.f};
    stream_stages<1>(ws, cursor, p.z1 != nullptr, st0, st1, 0, ARows<1>{operands, sums}, tot, [] { return 0; });
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
// weights again), and a set's 32-row weight tiles in units of 8 / S, S waves to a
// tile, each with a slice of the columns.  One workgroup fits a CU, and each takes
// an equal run of the units of all sets, so that no CU ends late because an expert
// has many pairs or because the chosen experts do not divide the chip; S is
// the one whose runs are shortest.  A workgroup finds its run from the ids itself
// (1.6 us; a launch of its own takes 4.5); a wave's weights are one stream through
// all its tiles.  In a build with time stamps a workgroup of the first product of 8 tokens
// has its activations in LDS 8 us after the start and streams until 50 us (median) to
// 62 us (those with a unit more).  Dividing only the last, partial turn of units into slices evens the
// ends out, but measured no faster (64 tokens: 165 + 103 against 161-173 + 91-102 us):
// the workgroups that are left have the memory to themselves.
constexpr int kWaves = 8, kSetPairs = 8, kMaxSets = 8;

struct Shared {
    uint8_t ring[kWaves][kRingBytes];
    uint8_t operands[kChunkOperands];
    float sums[kChunkSums];
    float part[2][kWaves][4][kWave];  // the slices' sums, of alternate units
    int expert[kMaxSets], count[kMaxSets];
    uint16_t pairs[kMaxSets][kSetPairs], tokens[kMaxSets][kSetPairs];
};
static_assert(sizeof(int) * kRouteMaxExperts + sizeof(uint16_t) * kMoePairs <= kChunkOperands,
              "the experts' counts and the ids lie in the operands' place");
static_assert(sizeof(Shared) <= 160 * 1024, "LDS");

struct Run {
    int q0, q1;      // units, counted through all sets
    int first_set;   // its sets are in Shared from here on
    int slices;      // S
    int units;       // of a set
};

// whole: A lies in LDS whole, so that waves can have unlike columns.  Everything
// here precedes the first weight, so dependent steps are kept few: the ids are
// read once, and what is divided is divided in lanes side by side.
__device__ __forceinline__ Run plan_run(const int32_t *ids, int P, int k, int E, int tiles, int stages, bool whole, Shared &s)
{
    constexpr int kThreads = kWaves * kWave, kEach = kMoePairs / kThreads;
    static_assert(kWaves == 8, "slices");
    int *cnt = reinterpret_cast<int *>(s.operands);
    uint16_t *chosen = reinterpret_cast<uint16_t *>(cnt + kRouteMaxExperts);
    const int t = threadIdx.x, lane = t % kWave, wave = t / kWave;
    int mine[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        mine[i] = i * kThreads + t < P ? ids[i * kThreads + t] : -1;
    for (int e = t; e < E; e += kThreads)
        cnt[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const bool live = mine[i] >= 0 && mine[i] < E;
        chosen[i * kThreads + t] = live ? (uint16_t)mine[i] : (uint16_t)0xffff;
        if (live)
            atomicAdd(&cnt[mine[i]], 1);
    }
    __syncthreads();
    int sets = 0;
    for (int c = 0; c < E; c += kWave)
        sets += c + lane < E ? (cnt[c + lane] + kSetPairs - 1) / kSetPairs : 0;
    sets = __builtin_amdgcn_readlane(wave_scan(sets), kWave - 1);
    // The longest run of units, in stages (doubled; joining slices costs about half
    // a stage): lane i has S = 2^i.
    const unsigned grid = gridDim.x;
    Run r;
    {
        const int log = lane % 4, S = 1 << log, units = (tiles * S + kWaves - 1) / kWaves;
        const int rounds = (int)(((unsigned)(sets * units) + grid - 1) / grid);
        int cost = rounds * (2 * ((stages + S - 1) >> log) + (S > 1 ? 1 : 0));
        if (S > 1 && (!whole || S > stages))
            cost = 0x7fffffff;
        int best = __builtin_amdgcn_readlane(cost, 0);
        r.slices = 1;
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const int c = __builtin_amdgcn_readlane(cost, i);
            if (c < best)
                best = c, r.slices = 1 << i;
        }
    }
    r.units = (tiles * r.slices + kWaves - 1) / kWaves;
    // At most 1152 sets of 2048 units, times 256 workgroups.
    const unsigned bound = (unsigned)(sets * r.units) * (blockIdx.x + (lane & 1)) / grid;
    r.q0 = __builtin_amdgcn_readlane((int)bound, 0);
    r.q1 = __builtin_amdgcn_readlane((int)bound, 1);
    const unsigned in_set = (unsigned)(lane & 1 ? r.q1 - 1 : r.q0) / (unsigned)r.units;
    r.first_set = __builtin_amdgcn_readlane((int)in_set, 0);
    const int last_set = __builtin_amdgcn_readlane((int)in_set, 1);
    // Wave i finds the run's i-th set: its expert, and its pairs in ascending order.
    const int set = r.first_set + wave;
    if (r.q0 < r.q1 && set <= last_set) {
        int before = 0, expert = 0, first = 0, count = 0;
        for (int c = 0; c < E; c += kWave) {
            const int n = c + lane < E ? cnt[c + lane] : 0, own = (n + kSetPairs - 1) / kSetPairs;
            const int v = wave_scan(own);
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
            const uint64_t mask = __ballot(chosen[c + lane] == expert);
            const int at = seen + __builtin_popcountll(mask & ((uint64_t(1) << lane) - 1));
            if ((mask >> lane & 1) && at >= 0 && at < kSetPairs)
                s.pairs[wave][at] = (uint16_t)(c + lane), s.tokens[wave][at] = (uint16_t)((c + lane) / k);
            seen += __builtin_popcountll(mask);
        }
        if (lane == 0)
            s.expert[wave] = expert, s.count[wave] = min(count, kSetPairs);
    }
    __syncthreads();
    return r;
}

// Cursor over a wave's tiles of a run: one in each unit, where there is one.
// A tile is kTileRows weight rows (of each kind).
template <int kTileRows>
struct RunCursor {
    const int *expert;
    int left, at;  // units to come, and the next one's place in its set, which is expert's first
    int units, per_unit, tiles, mine, st, st0, st1;
    __device__ __forceinline__ RunCursor(const Run &r, const Shared &s, int tiles_, int stages)
        : expert(s.expert), left(r.q1 - r.q0), at(r.q0 - r.first_set * r.units), units(r.units), tiles(tiles_)
    {
        // 1, 2, 4 or 8 slices.
        const int wave = threadIdx.x / kWave, log = __builtin_ctz(r.slices), slice = wave & (r.slices - 1);
        per_unit = kWaves >> log;
        mine = wave >> log;
        st0 = slice * stages >> log, st1 = (slice + 1) * stages >> log;
        st = st0;
    }
    __device__ __forceinline__ int tile(int place) const { return place * per_unit + mine; }
    __device__ __forceinline__ void step()
    {
        --left;
        if (++at == units)
            at = 0, ++expert;
    }
    __device__ __forceinline__ bool next(WeightStream<> &ws, int &stage)
    {
        if (st == st0) {
            while (left > 0 && tile(at) >= tiles)
                step();
            if (left <= 0)
                return false;
            ws.tile(__builtin_amdgcn_readfirstlane(*expert), tile(at) * kTileRows);
        }
        stage = st;
        if (++st == st1) {
            st = st0;
            step();
        }
        return true;
    }
};

// Units [q0, q1) of the run's set `set` against kRows rows of A.  With 16 rows, rows 8-15 are
// added to rows 0-7.  done(tile, sum) stores a tile's results and returns how many
// vector stores that is at least.
template <int kRows, class Cursor, class Load, class Done>
__device__ __forceinline__ void stream_set(WeightStream<> &ws, Cursor &cursor, const Run &r, bool zeros, int q0,
                                           int q1, int set, Shared &s, Load &&load, Done &&done)
{
    constexpr int kGroups = kChunkElems / 64 / kRows, kRegs = ARows<kRows>::kRegs;
    const int G = ws.G, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const ARows<kRows> A{s.operands, s.sums};
    const bool whole = G <= kGroups;
    float tot[kRegs], held[4];
    int held_tile = -1;
    const auto flush = [&] {
        const int stores = held_tile >= 0 ? done(held_tile, held) : 0;
        held_tile = -1;
        return stores;
    };
    for (int q = q0; q < q1; ++q) {
        const int tile = cursor.tile(q - (r.first_set + set) * r.units);
#pragma unroll
        for (int i = 0; i < kRegs; ++i)
            tot[i] = 0.f;
        for (int g0 = 0; g0 < G; g0 += kGroups) {
            if (!whole || q == q0)
                fill_rows<kRows, kWaves>(G, g0, s.operands, s.sums, load, [&] {
                    if (q == r.q0 && g0 == 0)
                        ws.start(cursor);
                });
            if (tile < cursor.tiles)
                stream_stages<kRows>(ws, cursor, zeros, max(cursor.st0, g0 / kStageGroups),
                                     min(cursor.st1, (g0 + kGroups) / kStageGroups), g0, A, tot, flush);
        }
        if constexpr (kRegs == 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tot[i] += tot[kRegs - 4 + i];
        if (r.slices > 1) {
            // Alternate units use alternate places: a place is written again only
            // after the barrier of the unit between.
            float(&part)[kWaves][4][kWave] = s.part[q % 2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[wave][i][lane] = tot[i];
            __syncthreads();
            if ((wave & (r.slices - 1)) == 0)
                for (int w = 1; w < r.slices; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tot[i] += part[wave + w][i][lane];
        }
        if (tile < cursor.tiles && (wave & (r.slices - 1)) == 0) {
            held_tile = tile;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                held[i] = tot[i];
        }
    }
    flush();
}

// The first product of many pairs: a tile is 16 hidden columns (their gate and up
// rows); A's rows are the set's tokens.
template <int kRows>
__device__ __forceinline__ void up_set(const UpArgs &p, WeightStream<> &ws, RunCursor<16> &cursor, const Run &r, int q0,
                                       int q1, int set, Shared &s)
{
    const int lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32, count = s.count[set];
    const auto load = [&](int row, int ch) {
        const int t = s.tokens[set][min(row, count - 1)];
        return __builtin_bit_cast(
            u32x4, act_order8(*reinterpret_cast<const u32x4 *>(p.x + (int64_t)t * p.ldx + ch * 8)));
    };
    const auto done = [&](int tile, const float(&tot)[4]) {
        int rows = count, column = l32;  // opaque: compared here, no masks kept through the stream
        asm volatile("" : "+v"(rows), "+v"(column));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = __shfl_xor(tot[i], 16);
            const int row = (kRows > 4 ? 4 * half : 0) + i;
            if (column < 16 && (kRows > 4 || half == 0) && row < rows)
                put_hidden(p.hidden, s.pairs[set][row], p.I, tile * 16 + l32, tot[i], u);
        }
        return 2 * min(4, count);  // of the lower half's rows at least
    };
    stream_set<kRows>(ws, cursor, r, p.z1 != nullptr, q0, q1, set, s, load, done);
}

__global__ __launch_bounds__(kWaves * kWave, 2) void moe_up_kernel(const UpArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int tiles = p.I / 16;
    WeightStream<> ws(p.w1, p.s1, p.z1, 2 * p.I, p.H / 64, p.I, s.ring[threadIdx.x / kWave]);
    const Run r = plan_run(p.r.ids, p.P, p.k, p.E, tiles, ws.stages(), p.H * kSetPairs <= kChunkElems, s);
    RunCursor<16> cursor(r, s, tiles, ws.stages());
    int q = r.q0;
    for (int set = 0; q < r.q1; ++set) {
        const int end = min(r.q1, (r.first_set + set + 1) * r.units);
        if (s.count[set] <= 4)
            up_set<4>(p, ws, cursor, r, q, end, set, s);
        else
            up_set<8>(p, ws, cursor, r, q, end, set, s);
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

constexpr int kFewWaves = 8, kFewDepth = 3;
__host__ __device__ constexpr int few_half(int groups) { return stage_groups((groups + 1) / 2); }
constexpr int few_down_lds(int P, int G)
{
    return kFewWaves * (kFewDepth * kStageBytes + few_half(G) * (512 + 16)) + (P > kFewWaves ? P : kFewWaves) * 64;
}

// Few pairs: a workgroup owns 16 output columns (so that the columns spread over
// the chip); its waves take the pairs (or slices of the I columns, where there are
// fewer pairs than waves), then every output adds its token's slots in order.
// A tile's 32 rows are the 16 columns' weights of the first and of the second half
// of the I columns; A's four rows are the pair's first and second parts of the
// first half, then of the second.  A is the wave's own: no barriers until the end.
__global__ __launch_bounds__(kFewWaves * kWave) void moe_down_few_kernel(const DownArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // rings, operands, group sums, results
    __shared__ int s_id[kMoeFewPairs];
    __shared__ float s_weight[kMoeFewPairs];
    const int I = p.I, G = I / 64, P = p.T * p.k;
    const int n0 = xcd_block(blockIdx.x, gridDim.x) * 16;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, l32 = lane % 32;
    const int GH = (G + 1) / 2, GP = few_half(G), stages = GP / kStageGroups;
    const int slices = max(1, min(kFewWaves / P, stages));
    constexpr int kRing = kFewDepth * kStageBytes;
    uint8_t *operands = smem + kFewWaves * kRing + wave * GP * 512;                           // [GP][4][2][4] x 16 bytes
    float *sums = reinterpret_cast<float *>(smem + kFewWaves * (kRing + GP * 512)) + wave * GP * 4;  // [GP][4]
    float *s_sum = reinterpret_cast<float *>(smem + kFewWaves * (kRing + GP * 528));          // [slices][P][16]

    WeightStream<kFewDepth> ws(p.w2, p.s2, p.z2, p.H, G, 0, smem + wave * kRing);
    const int id = threadIdx.x < P ? p.ids[threadIdx.x] : 0;
    const float weight = threadIdx.x < P ? p.weights[threadIdx.x] : 0.f;
    for (int it = wave; it < P * slices; it += kFewWaves) {
        const int pr = it / slices, sl = it - pr * slices;
        const int e = __builtin_amdgcn_readfirstlane(p.ids[pr]);
        if (e < 0 || e >= p.E)
            continue;
        const int st0 = sl * stages / slices, st1 = (sl + 1) * stages / slices;
        OneTile cursor{st0, st1};
        ws.tile(e, n0);
        // A's loads, then the weights (loads retire in order), then A to LDS: two
        // stages' chunks of the four rows at a time.
        bool started = false;
        for (int ch0 = st0 * kStageGroups * 8; ch0 < st1 * kStageGroups * 8; ch0 += kWave) {
            const int ch = ch0 + lane;
            u32x4 v[4];
#pragma unroll
            for (int row = 0; row < 4; ++row) {
                const int col = ch + row / 2 * GH * 8;
                v[row] = u32x4{0u, 0u, 0u, 0u};
                if (ch < GH * 8 && col < G * 8)
                    v[row] = *reinterpret_cast<const u32x4 *>(p.hidden + ((int64_t)pr * 2 + row % 2) * I + col * 8);
            }
            if (!started) {
                __builtin_amdgcn_sched_barrier(0);
                ws.start(cursor);
                __builtin_amdgcn_sched_barrier(0);
                started = true;
            }
            if (ch < st1 * kStageGroups * 8)
#pragma unroll
                for (int row = 0; row < 4; ++row)
                    put_chunk<4>(operands, sums, row, ch, __builtin_bit_cast(u32x4, act_order8(v[row])));
        }
        wait_lds();
        const ARows<4> A{operands, sums};
        float tot[4] = {0.f, 0.f, 0.f, 0.f};
        stream_stages<4>(ws, cursor, p.z2 != nullptr, st0, st1, 0, A, tot, [] { return 0; });
        float v = l32 < 16 ? tot[0] + tot[1] : tot[2] + tot[3];
        v += __shfl_xor(v, 16);
        if (lane < 16)
            s_sum[(sl * P + pr) * 16 + lane] = v;
    }
    if (threadIdx.x < P)
        s_id[threadIdx.x] = id, s_weight[threadIdx.x] = weight;
    __syncthreads();
    for (int o = threadIdx.x; o < p.T * 16; o += kFewWaves * kWave) {
        const int t = o / 16, col = o % 16;
        float y = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const int pr = t * p.k + j;
            if (s_id[pr] >= 0 && s_id[pr] < p.E) {
                float v = s_sum[pr * 16 + col];
                for (int sl = 1; sl < slices; ++sl)
                    v += s_sum[(sl * P + pr) * 16 + col];
                y = __builtin_fmaf(s_weight[pr], v, y);
            }
        }
        p.out[(int64_t)t * p.ldo + n0 + col] = f32_to_bf16(y);
    }
}

// The second product of many pairs: a tile is 32 output columns, A's rows are the
// first parts of the set's pairs, then the second parts; the sums of each pair go
// to moe_combine_kernel.
template <int kPairs>
__device__ __forceinline__ void down_set(const DownArgs &p, WeightStream<> &ws, RunCursor<32> &cursor, const Run &r, int q0,
                                         int q1, int set, Shared &s)
{
    constexpr int kRows = 2 * kPairs;
    const int lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32, count = s.count[set];
    const auto load = [&](int row, int ch) {
        const int pr = s.pairs[set][min(row % kPairs, count - 1)];
        return __builtin_bit_cast(u32x4, act_order8(*reinterpret_cast<const u32x4 *>(
                                             p.hidden + ((int64_t)pr * 2 + row / kPairs) * p.I + ch * 8)));
    };
    const auto done = [&](int tile, const float(&tot)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // Of four pairs the second parts are in the other half of the wave.
            const float v = kPairs == 4 ? tot[i] + __shfl_xor(tot[i], 32) : tot[i];
            const int at = kPairs == 4 ? i : 4 * half + i;
            if (at < count && (kPairs > 4 || half == i / 2))
                p.y[(int64_t)s.pairs[set][at] * p.H + tile * 32 + l32] = v;
        }
        return min(4, count);
    };
    stream_set<kRows>(ws, cursor, r, p.z2 != nullptr, q0, q1, set, s, load, done);
}

__global__ __launch_bounds__(kWaves * kWave, 2) void moe_down_kernel(const DownArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int tiles = p.H / 32;
    WeightStream<> ws(p.w2, p.s2, p.z2, p.H, p.I / 64, 16, s.ring[threadIdx.x / kWave]);
    const Run r = plan_run(p.ids, p.T * p.k, p.k, p.E, tiles, ws.stages(), p.I * 2 * kSetPairs <= kChunkElems, s);
    RunCursor<32> cursor(r, s, tiles, ws.stages());
    int q = r.q0;
    for (int set = 0; q < r.q1; ++set) {
        const int end = min(r.q1, (r.first_set + set + 1) * r.units);
        if (s.count[set] <= 4)
            down_set<4>(p, ws, cursor, r, q, end, set, s);
        else
            down_set<8>(p, ws, cursor, r, q, end, set, s);
        q = end;
    }
}

// out[t] = sum over the slots, in order; four columns a thread, a token a grid row.
// Eight slots' loads are in flight at a time, and wait for no id: an empty slot's
// results are in the workspace too, and not used.
__global__ __launch_bounds__(64) void moe_combine_kernel(const DownArgs p)
{
    const int t = blockIdx.y, n = (blockIdx.x * 64 + threadIdx.x) * 4;
    if (n >= p.H)
        return;
    v4f y = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        v4f v[8];
        float w[8];
        bool live[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int pr = t * p.k + min(j0 + j, p.k - 1), e = p.ids[pr];
            live[j] = j0 + j < p.k && e >= 0 && e < p.E;
            w[j] = p.weights[pr];
            v[j] = *reinterpret_cast<const v4f *>(p.y + (int64_t)pr * p.H + n);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (live[j])
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = __builtin_fmaf(w[j], v[j][i], y[i]);
    }
    *reinterpret_cast<u32x2 *>(p.out + (int64_t)t * p.ldo + n) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

// More than 64 KiB of dynamic LDS needs the kernel's attribute raised once; a
// kernel's static LDS counts against the CU's 160 KiB too.
constexpr int kMaxLds = 160 * 1024, kCus = 256;
template <auto kernel, int bytes = kMaxLds>
hipError_t allow_lds()
{
    static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e;
}

template <int kNe, bool kBf16>
hipError_t launch_up_few(const UpArgs &a, hipStream_t s)
{
    constexpr auto kernel = moe_up_few_kernel<kNe, kBf16>;
    const hipError_t e = allow_lds<kernel, kMaxLds - 1024>();
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
    return with_lane_logits(a.E, [&](auto ne) {
        return a.r.bf16 ? launch_up_few<decltype(ne)::value, true>(a, s) : launch_up_few<decltype(ne)::value, false>(a, s);
    });
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

    static_assert(few_down_lds(kMoeFewPairs, kMoeFewInner / 64) <= kMaxLds - 1024, "LDS");
    const bool few = P <= kMoeFewPairs && w.I <= kMoeFewInner;
    if (r.logits && !few) {
        const int e = launch_moe_route(r.logits, r.bf16, T, w.E, r.ldl, r.k, r.renormalize, r.ids, r.weights, stream);
        if (e != 0)
            return e;
    }
    const UpArgs ua{x, ldx, r.k, w.w1, w.s1, w.z1, w.E, w.H, w.I, P, r, hidden};
    // One workgroup a CU, and no more than there can be units.  A run has at most
    // kMaxSets sets: 256 runs of up to 1152 sets, or less than a unit each.
    const int64_t most_sets = (w.E < P ? w.E : P) + P / kSetPairs;
    const auto grid = [&](int tiles) { return most_sets * tiles < kCus ? (int)most_sets * tiles : kCus; };
    hipError_t e = launch_up(ua, few, grid(w.I / 16), s);
    if (e != hipSuccess)
        return (int)e;
    const DownArgs da{hidden, w.w2, w.s2, w.z2, w.E, w.H, w.I, T, r.k, r.ids, r.weights, y, out, ldo};
    if (few) {
        e = allow_lds<moe_down_few_kernel, kMaxLds - 1024>();
        if (e != hipSuccess)
            return (int)e;
        hipLaunchKernelGGL(moe_down_few_kernel, dim3(w.H / 16), dim3(kFewWaves * kWave), few_down_lds(P, w.I / 64), s,
                           da);
    } else {
        e = allow_lds<moe_down_kernel>();
        if (e != hipSuccess)
            return (int)e;
        hipLaunchKernelGGL(moe_down_kernel, dim3(grid(w.H / 32)), dim3(kWaves * kWave), sizeof(Shared), s, da);
        hipLaunchKernelGGL(moe_combine_kernel, dim3((w.H / 4 + 63) / 64, T), dim3(64), 0, s, da);
    }
    return (int)hipGetLastError();
}

}  // namespace ck
