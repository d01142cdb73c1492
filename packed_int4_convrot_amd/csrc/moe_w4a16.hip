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

// The expert of unit y of a launch over min(E, P) units, and its pairs in
// ascending order.  With more experts than pairs, unit y is pair y's expert, if
// y is the first pair to choose it.  count 0: nothing to do.
struct Picked {
    int expert, count;
};
__device__ __forceinline__ Picked pick(const int32_t *ids, int P, int E, int y, uint16_t *s_list)
{
    const int lane = threadIdx.x % kWave;
    const bool writes = threadIdx.x < kWave;
    const int e = E <= P ? y : __builtin_amdgcn_readfirstlane(ids[y]);
    Picked r{e, 0};
    if (e < 0 || e >= E)
        return r;
    int first = -1;
    for (int c = 0; c < P; c += kWave) {
        const int v = c + lane < P ? ids[c + lane] : -1;
        const uint64_t mask = __ballot(v == e);
        if (mask) {
            if (first < 0)
                first = c + __builtin_ctzll(mask);
            if (writes && v == e)
                s_list[r.count + __builtin_popcountll(mask & ((uint64_t(1) << lane) - 1))] = (uint16_t)(c + lane);
            r.count += __builtin_popcountll(mask);
        }
    }
    if (E > P && first != y)
        r.count = 0;
    return r;
}

// ---------------------------------------------------------------- first product

constexpr int kWaves = 4;

struct UpArgs {
    const uint16_t *x;
    int64_t ldx;
    int k;
    const uint8_t *w1;
    const uint16_t *s1, *z1;
    int E, H, I, P;
    MoeRouting r;
    uint16_t *hidden;         // [P][2][I]: first parts, second parts, in operand order
};

// silu(g) u of hidden column n of a pair, as two bf16.
__device__ __forceinline__ void put_hidden(uint16_t *hidden, int pair, int I, int n, float g, float u)
{
    uint16_t hi, lo;
    split_bf16(g / (1.f + expf(-g)) * u, hi, lo);
    uint16_t *dst = hidden + (int64_t)pair * 2 * I + n / 8 * 8 + act_slot8(n % 8);
    dst[0] = hi;
    dst[I] = lo;
}

// Few pairs.  A unit is a pair, routed here (kNe logits a lane) or by the given
// ids (kNe 0); a workgroup owns 16 hidden columns of it, a wave's tile being
// their 16 gate and 16 up rows, and the waves split the H columns.
template <int kNe, bool kBf16>
__global__ __launch_bounds__(kWaves * kWave) void moe_up_few_kernel(const UpArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // rings, operands, sums
    __shared__ float s_red[kWaves][32];
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
    const int st0 = wave * stages / kWaves, st1 = (wave + 1) * stages / kWaves;
    const WeightStream ws(p.w1, p.s1, p.z1, e, 2 * I, G, n0, I, smem + wave * kRingBytes);
#pragma unroll
    for (int i = 0; i < kStages; ++i)
        if (st0 + i < st1)
            ws.issue(st0 + i);
    uint8_t *operands = smem + kWaves * kRingBytes;
    const int GP = stage_groups(G);
    float *sums = reinterpret_cast<float *>(operands + GP * 128);
    const uint16_t *x = p.x + (int64_t)t * p.ldx;
    for (int c = threadIdx.x; c < GP * 8; c += kWaves * kWave) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (c < G * 8)
            v = __builtin_bit_cast(u32x4, act_order8(*reinterpret_cast<const u32x4 *>(x + c * 8)));
        put_chunk<1>(operands, sums, 0, c, v);
    }
    __syncthreads();
    float tot[1] = {0.f};
    stream_stages<1>(ws, p.z1 != nullptr, st0, st1, st1, 0, ARows<1>{operands, sums}, tot);
    if (lane < 32)
        s_red[wave][l32] = tot[0];
    __syncthreads();
    if (threadIdx.x < 16) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            g += s_red[w][l32], u += s_red[w][l32 + 16];
        put_hidden(p.hidden, y, I, n0 + l32, g, u);
    }
}

// Otherwise: a workgroup owns 64 hidden columns of one expert, 16 a wave (their
// gate and up rows), for tiles of kRows of its pairs.
struct Shared {
    uint8_t ring[kWaves][kRingBytes];
    uint8_t operands[kChunkOperands];
    float sums[kChunkElems / 64];
    uint16_t list[kMoePairs];
};

template <int kRows>
__device__ __forceinline__ void up_tile(const UpArgs &p, const Picked &pk, int p0, int n0, Shared &s)
{
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32;
    const WeightStream ws(p.w1, p.s1, p.z1, pk.expert, 2 * p.I, p.H / 64, n0, p.I, s.ring[wave]);
    float tot[ARows<kRows>::kRegs];
#pragma unroll
    for (int i = 0; i < ARows<kRows>::kRegs; ++i)
        tot[i] = 0.f;
    const auto load = [&](int row, int ch) {
        const int pr = s.list[min(p0 + row, pk.count - 1)];
        return __builtin_bit_cast(
            u32x4, act_order8(*reinterpret_cast<const u32x4 *>(p.x + (int64_t)(pr / p.k) * p.ldx + ch * 8)));
    };
    stream_rows<kRows, kWaves>(ws, p.z1 != nullptr, true, s.operands, s.sums, load, tot);
#pragma unroll
    for (int i = 0; i < ARows<kRows>::kRegs; ++i) {
        const float u = __shfl_xor(tot[i], 16);
        const int row = i / 4 * 8 + 4 * half + i % 4;
        if (l32 < 16 && row < kRows && p0 + row < pk.count)
            put_hidden(p.hidden, s.list[p0 + row], p.I, n0 + l32, tot[i], u);
    }
}

__global__ __launch_bounds__(kWaves * kWave, 2) void moe_up_kernel(const UpArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int tiles = p.I / 64, y = blockIdx.x / tiles;
    const Picked pk = pick(p.r.ids, p.P, p.E, y, s.list);
    if (pk.count == 0)
        return;
    __syncthreads();  // list
    const int n0 = blockIdx.x % tiles * 64 + threadIdx.x / kWave * 16;
    for (int p0 = 0; p0 < pk.count;) {
        const int left = pk.count - p0;
        if (left <= 4)
            up_tile<4>(p, pk, p0, n0, s), p0 += 4;
        else if (left <= 8)
            up_tile<8>(p, pk, p0, n0, s), p0 += 8;
        else
            up_tile<16>(p, pk, p0, n0, s), p0 += 16;
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
            v = *reinterpret_cast<const u32x4 *>(p.hidden + (int64_t)row * I + ch * 8);
        put_chunk<1>(operands, sums, 0, c, v);
    }
    __syncthreads();
    for (int it = wave; it < P * slices; it += kFewWaves) {
        const int pr = it / slices, sl = it % slices;
        const int e = __builtin_amdgcn_readfirstlane(p.ids[pr]);
        if (e < 0 || e >= p.E)
            continue;
        const int st0 = sl * stages / slices, st1 = (sl + 1) * stages / slices;
        const WeightStream ws(p.w2, p.s2, p.z2, e, H, G, n0, 16, smem + wave * kRingBytes);
        wait_lds();  // the ring's last operands have been read
#pragma unroll
        for (int i = 0; i < kStages; ++i)
            if (st0 + i < st1)
                ws.issue(st0 + i);
        float tot[1] = {0.f};
        stream_stages<1>(ws, p.z2 != nullptr, st0, st1, st1, 0,
                         ARows<1>{operands + (2 * pr + l32 / 4 % 2) * GP * 128, sums + (2 * pr + half) * GP}, tot);
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

// Otherwise: a workgroup owns 128 output columns (32 a wave) of one expert and
// writes the sums of its pairs, which moe_combine_kernel adds.  A's rows are the
// first parts of a tile's pairs, then the second parts.
template <int kPairs>
__device__ __forceinline__ void down_tile(const DownArgs &p, const Picked &pk, int p0, int n0, Shared &s)
{
    constexpr int kRows = 2 * kPairs, kRegs = ARows<kRows>::kRegs;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, l32 = lane % 32, half = lane / 32;
    const bool live = n0 < p.H;
    const WeightStream ws(p.w2, p.s2, p.z2, pk.expert, p.H, p.I / 64, live ? n0 : 0, 16, s.ring[wave]);
    float tot[kRegs];
#pragma unroll
    for (int i = 0; i < kRegs; ++i)
        tot[i] = 0.f;
    const auto load = [&](int row, int ch) {
        const int pr = s.list[min(p0 + row % kPairs, pk.count - 1)];
        return *reinterpret_cast<const u32x4 *>(p.hidden + ((int64_t)pr * 2 + row / kPairs) * p.I + ch * 8);
    };
    stream_rows<kRows, kWaves>(ws, p.z2 != nullptr, live, s.operands, s.sums, load, tot);
    if (!live)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // The second parts are in the other half of the wave (4 pairs) or the other four registers (8).
        const float v = kPairs == 4 ? tot[i] + __shfl_xor(tot[i], 32) : tot[i] + tot[kRegs - 4 + i];
        const int at = kPairs == 4 ? i : 4 * half + i;
        if (p0 + at < pk.count && (kPairs > 4 || half == i / 2))
            p.y[(int64_t)s.list[p0 + at] * p.H + n0 + l32] = v;
    }
}

__global__ __launch_bounds__(kWaves * kWave, 2) void moe_down_kernel(const DownArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int tiles = (p.H + 32 * kWaves - 1) / (32 * kWaves);
    const Picked pk = pick(p.ids, p.T * p.k, p.E, blockIdx.x / tiles, s.list);
    if (pk.count == 0)
        return;
    __syncthreads();  // list
    const int n0 = (blockIdx.x % tiles * kWaves + threadIdx.x / kWave) * 32;
    for (int p0 = 0; p0 < pk.count;) {
        const int left = pk.count - p0;
        if (left <= 4)
            down_tile<4>(p, pk, p0, n0, s), p0 += 4;
        else
            down_tile<8>(p, pk, p0, n0, s), p0 += 8;
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
constexpr int kMaxLds = 150 * 1024;
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
    const int lds = kWaves * kRingBytes + stage_groups(a.H / 64) * (128 + 4);
    hipLaunchKernelGGL(kernel, dim3((runs + kXcds - 1) / kXcds * kXcds * 4), dim3(kWaves * kWave), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_up(const UpArgs &a, bool few, int units, hipStream_t s)
{
    if (!few) {
        const hipError_t e = allow_lds<moe_up_kernel>();
        if (e != hipSuccess)
            return e;
        hipLaunchKernelGGL(moe_up_kernel, dim3(units * (a.I / 64)), dim3(kWaves * kWave), sizeof(Shared), s, a);
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
    const int units = w.E < P ? w.E : P;
    const UpArgs ua{x, ldx, r.k, w.w1, w.s1, w.z1, w.E, w.H, w.I, P, r, hidden};
    hipError_t e = launch_up(ua, few, units, s);
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
        const int tiles = (w.H + 32 * kWaves - 1) / (32 * kWaves);
        hipLaunchKernelGGL(moe_down_kernel, dim3(units * tiles), dim3(kWaves * kWave), sizeof(Shared), s, da);
        const int64_t quads = (int64_t)T * (w.H / 4);
        hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s, da);
    }
    return (int)hipGetLastError();
}

}  // namespace ck
