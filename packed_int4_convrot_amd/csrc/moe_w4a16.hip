// Mixture-of-experts layer on packed uint4 experts (AWQ W4A16) for few tokens.
//
//   W[n, c] = (q - 8) s[c / 64, n] + z[c / 64, n], kept exact,
//   h = silu(W1[e][:I] x) * (W1[e][I:] x),  y = W2[e] h,
//   out[t] = sum over the token's slots j of weight_j y_{e_j}.
//
// Three launches: the plan (routing, then the (token, slot) pairs sorted by
// expert), the first product with the gate, the second with the weighted sum.
// Few tokens make this a matter of streaming the chosen experts' weights once,
// so every kernel multiplies on the 16 x 16 bf16 MFMA whatever the number of
// tokens and the weights go straight to registers.  Per 64-column group g,
//   sum_c x_c W[n, c] = s P + (z - 136 s) X,  P = sum x_c (128 + q_c), X = sum x_c,
// where bf16(128 + q) costs an and-or per pair of codes, and X comes from an
// MFMA against ones in the register layout that P has.  Sums are fp32.
#include "moe_route.h"
#include "rows_launch.h"

namespace ck {
namespace {

struct Chosen {
    int expert, first, count, pad;
};
__device__ __forceinline__ const Chosen *plan_records(const int *plan)
{
    return reinterpret_cast<const Chosen *>(plan + 4);
}

constexpr int kPlanThreads = 1024;

// One workgroup: routes the tokens (a wave each) or reads given ids, then
// sorts the pairs by expert.  The order of an expert's pairs is that of the
// LDS atomics; no result depends on it, since a pair's sums do not depend on
// which row of which tile it takes.
template <int kNe, bool kBf16, bool kRoute>
__global__ __launch_bounds__(kPlanThreads) void moe_plan_kernel(const void *__restrict__ logits, int T, int E,
                                                                int64_t ldl, int k, bool renormalize,
                                                                int32_t *__restrict__ ids,
                                                                float *__restrict__ weights,
                                                                int *__restrict__ plan)
{
    __shared__ int s_id[kMoePairs];
    __shared__ int s_count[kRouteMaxExperts];
    __shared__ int s_start[kRouteMaxExperts];
    __shared__ int s_wave[kPlanThreads / kWave];
    const int t = threadIdx.x, lane = t % kWave, wave = t / kWave;
    const int P = T * k;
    s_count[t] = 0;
    if constexpr (kRoute) {
#pragma unroll 1
        for (int tok = wave; tok < T; tok += kPlanThreads / kWave) {
            int id;
            float w;
            route_row<kNe, kBf16>(static_cast<const uint8_t *>(logits) + (int64_t)tok * ldl * (kBf16 ? 2 : 4), E, k,
                                  renormalize, lane, id, w);
            if (lane < k) {
                s_id[tok * k + lane] = id;
                ids[tok * k + lane] = id;
                weights[tok * k + lane] = w;
            }
        }
    } else {
        if (t < P)
            s_id[t] = ids[t];
    }
    __syncthreads();
    int e = -1, at = 0;
    if (t < P) {
        e = s_id[t];
        if (e < 0 || e >= E)
            e = -1;
        else
            at = atomicAdd(&s_count[e], 1);
    }
    __syncthreads();
    // Exclusive scan over the experts of (chosen, pairs) as two 16-bit halves.
    const int c = s_count[t];
    int v = (c > 0 ? 1 << 16 : 0) + c;
    const int own = v;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d)
            v += u;
    }
    if (lane == kWave - 1)
        s_wave[wave] = v;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / kWave; ++w) {
        if (w < wave)
            before += s_wave[w];
        total += s_wave[w];
    }
    const int excl = before + v - own;
    s_start[t] = excl & 0xffff;
    Chosen *rec = reinterpret_cast<Chosen *>(plan + 4);
    if (c > 0)
        rec[excl >> 16] = Chosen{t, excl & 0xffff, c, 0};
    if (t == 0)
        plan[0] = total >> 16;
    __syncthreads();
    int *pairs = plan + 4 + 4 * min(E, P);
    if (e >= 0)
        pairs[s_start[e] + at] = t;
}

// ---------------------------------------------------------------- first product

constexpr int kUpWaves = 4;
constexpr int kUpAhead = 4;  // groups per load batch

// A workgroup owns 16 hidden columns (16 gate rows and 16 up rows) of one
// chosen expert; its waves split the H columns and are summed through LDS.
// Neighbouring column tiles share lines of the scales, so runs of four tiles
// go to one XCD, and the runs go round the XCDs (the chosen experts come first).
__global__ __launch_bounds__(kUpWaves * kWave) void moe_up_kernel(
    const uint16_t *__restrict__ x, int64_t ldx, int k, const uint8_t *__restrict__ w1,
    const uint16_t *__restrict__ s1, const uint16_t *__restrict__ z1, int H, int I, const int *__restrict__ plan,
    int records, uint16_t *__restrict__ hidden)
{
    __shared__ float s_red[kUpWaves][2][256];
    const int tiles = I / 16;
    const int local = blockIdx.x / kXcds;
    const int unit = (local / 4) * kXcds + blockIdx.x % kXcds;
    const int a = unit / (tiles / 4), n0 = (unit % (tiles / 4) * 4 + local % 4) * 16;
    if (a >= plan[0])
        return;
    const Chosen ch = plan_records(plan)[a];
    const int *pairs = plan + 4 + 4 * records;

    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int l16 = lane % 16, quarter = lane / 16;
    const int G = H / 64;
    const int g0 = wave * G / kUpWaves, g1 = (wave + 1) * G / kUpWaves;
    const uint8_t *wrow[2];
    const uint16_t *srow[2], *zrow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int n = j * I + n0 + l16;
        wrow[j] = w1 + ((int64_t)ch.expert * 2 * I + n) * (H / 2) + 8 * quarter;
        srow[j] = s1 + (int64_t)ch.expert * G * 2 * I + n;
        zrow[j] = z1 ? z1 + (int64_t)ch.expert * G * 2 * I + n : nullptr;
    }
    const v8bf ones = bf16_ones();

    for (int p0 = 0; p0 < ch.count; p0 += 16) {
        const int pr = pairs[ch.first + min(p0 + l16, ch.count - 1)];
        const uint16_t *xrow = x + (int64_t)(pr / k) * ldx + 16 * quarter;
        v4f tot[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        for (int gb = g0; gb < g1; gb += kUpAhead) {
            u32x2 w[kUpAhead][2];
            u32x4 xv[kUpAhead][2];
            uint32_t sv[kUpAhead][2], zv[kUpAhead][2];
#pragma unroll
            for (int u = 0; u < kUpAhead; ++u) {
                const int g = min(gb + u, g1 - 1);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    w[u][j] = *reinterpret_cast<const u32x2 *>(wrow[j] + g * 32);
                    sv[u][j] = srow[j][(int64_t)g * 2 * I];
                    zv[u][j] = z1 ? zrow[j][(int64_t)g * 2 * I] : 0;
                    xv[u][j] = *reinterpret_cast<const u32x4 *>(xrow + g * 64 + 8 * j);
                }
            }
#pragma unroll
            for (int u = 0; u < kUpAhead; ++u) {
                if (gb + u < g1) {
                    const v8bf x0 = act_order8(xv[u][0]), x1 = act_order8(xv[u][1]);
                    const v4f zero = {0.f, 0.f, 0.f, 0.f};
                    const v4f X = mfma16(x1, ones, mfma16(x0, ones, zero));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const v4f acc = mfma16(x1, w4_bf16_plus128(w[u][j][1]),
                                               mfma16(x0, w4_bf16_plus128(w[u][j][0]), zero));
                        const float s = bf16_to_f32(sv[u][j]);
                        const float zc = __builtin_fmaf(-136.f, s, bf16_to_f32(zv[u][j]));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tot[j][i] = __builtin_fmaf(s, acc[i], __builtin_fmaf(zc, X[i], tot[j][i]));
                    }
                }
            }
        }
        __syncthreads();  // the previous tile's sums have been read
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s_red[wave][j][i * kWave + lane] = tot[j][i];
        __syncthreads();
        const int row = threadIdx.x / 16, col = threadIdx.x % 16;
        if (p0 + row < ch.count) {
            const int at = (row % 4) * kWave + (row / 4) * 16 + col;
            float g = s_red[0][0][at], u = s_red[0][1][at];
#pragma unroll
            for (int w = 1; w < kUpWaves; ++w)
                g += s_red[w][0][at], u += s_red[w][1][at];
            const float h = g / (1.f + expf(-g)) * u;
            uint16_t hi, lo;
            split_bf16(h, hi, lo);
            // Per eight columns: 8 first parts, then 8 second parts, in MFMA order.
            uint16_t *dst = hidden + (int64_t)(ch.first + p0 + row) * 2 * I + (n0 + col) / 8 * 16 + act_slot8(col % 8);
            dst[0] = hi;
            dst[8] = lo;
        }
    }
}

// --------------------------------------------------------------- second product

constexpr int kDownWaves = 8;
constexpr int kDownAhead = 4;

// A workgroup owns 16 output columns of every token.  Its waves take the
// chosen experts (or slices of the I columns, where there are fewer experts than
// waves) in turn and leave one sum per pair and slice in LDS; then each output
// adds its token's slots in order.  A tile is eight pairs: the first parts of
// h are its rows 0-7, the second parts its rows 8-15, added at the end.
__global__ __launch_bounds__(kDownWaves * kWave) void moe_down_kernel(
    const uint16_t *__restrict__ hidden, const uint8_t *__restrict__ w2, const uint16_t *__restrict__ s2,
    const uint16_t *__restrict__ z2, int H, int I, int T, int k, int E, const int *__restrict__ plan, int records,
    const int32_t *__restrict__ ids, const float *__restrict__ weights, uint16_t *__restrict__ out, int64_t ldo)
{
    extern __shared__ float s_sum[];  // [slices][pairs][16]
    const int n0 = xcd_block(blockIdx.x, gridDim.x) * 16;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int l16 = lane % 16, quarter = lane / 16;
    const int P = T * k, G = I / 64;
    const int A = plan[0];
    const int *pairs = plan + 4 + 4 * records;
    const int slices = A > 0 ? max(1, min(min(kDownWaves / A, kMoePairs / P), G)) : 1;
    const v8bf ones = bf16_ones();

    for (int it = wave; it < A * slices; it += kDownWaves) {
        const int sl = it % slices;
        const Chosen ch = plan_records(plan)[it / slices];
        const int g0 = sl * G / slices, g1 = (sl + 1) * G / slices;
        const uint8_t *wrow = w2 + ((int64_t)ch.expert * H + n0 + l16) * (I / 2) + 8 * quarter;
        const uint16_t *srow = s2 + (int64_t)ch.expert * G * H + n0 + l16;
        const uint16_t *zrow = z2 ? z2 + (int64_t)ch.expert * G * H + n0 + l16 : nullptr;
        for (int p0 = 0; p0 < ch.count; p0 += 8) {
            const uint16_t *hrow = hidden + (int64_t)(ch.first + min(p0 + l16 % 8, ch.count - 1)) * 2 * I +
                                   32 * quarter + (l16 >= 8 ? 8 : 0);
            v4f tot = {0.f, 0.f, 0.f, 0.f};
            for (int gb = g0; gb < g1; gb += kDownAhead) {
                u32x2 w[kDownAhead];
                u32x4 hv[kDownAhead][2];
                uint32_t sv[kDownAhead], zv[kDownAhead];
#pragma unroll
                for (int u = 0; u < kDownAhead; ++u) {
                    const int g = min(gb + u, g1 - 1);
                    w[u] = *reinterpret_cast<const u32x2 *>(wrow + g * 32);
                    sv[u] = srow[(int64_t)g * H];
                    zv[u] = z2 ? zrow[(int64_t)g * H] : 0;
                    hv[u][0] = *reinterpret_cast<const u32x4 *>(hrow + g * 128);
                    hv[u][1] = *reinterpret_cast<const u32x4 *>(hrow + g * 128 + 16);
                }
#pragma unroll
                for (int u = 0; u < kDownAhead; ++u) {
                    if (gb + u < g1) {
                        const v8bf h0 = __builtin_bit_cast(v8bf, hv[u][0]), h1 = __builtin_bit_cast(v8bf, hv[u][1]);
                        const v4f zero = {0.f, 0.f, 0.f, 0.f};
                        const v4f X = mfma16(h1, ones, mfma16(h0, ones, zero));
                        const v4f acc =
                            mfma16(h1, w4_bf16_plus128(w[u][1]), mfma16(h0, w4_bf16_plus128(w[u][0]), zero));
                        const float s = bf16_to_f32(sv[u]);
                        const float zc = __builtin_fmaf(-136.f, s, bf16_to_f32(zv[u]));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tot[i] = __builtin_fmaf(s, acc[i], __builtin_fmaf(zc, X[i], tot[i]));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = tot[i] + __shfl_xor(tot[i], 32);
                const int row = p0 + 4 * quarter + i;
                if (quarter < 2 && row < ch.count)
                    s_sum[((int64_t)sl * P + pairs[ch.first + row]) * 16 + l16] = y;
            }
        }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < T * 16; o += kDownWaves * kWave) {
        const int t = o / 16, col = o % 16;
        float y = 0.f;
        for (int j = 0; j < k; ++j) {
            const int p = t * k + j, e = ids[p];
            if (e >= 0 && e < E) {
                float v = s_sum[p * 16 + col];
                for (int sl = 1; sl < slices; ++sl)
                    v += s_sum[(sl * P + p) * 16 + col];
                y = __builtin_fmaf(weights[p], v, y);
            }
        }
        out[(int64_t)t * ldo + n0 + col] = f32_to_bf16(y);
    }
}

template <bool kBf16>
void launch_plan(const MoeRouting &r, int T, int E, int *plan, hipStream_t s)
{
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(1), dim3(kPlanThreads), 0, s, r.logits, T, E, r.ldl, r.k, r.renormalize,
                           r.ids, r.weights, plan);
    };
    if (!r.logits)
        go(moe_plan_kernel<1, false, false>);
    else if (E <= 64)
        go(moe_plan_kernel<1, kBf16, true>);
    else if (E <= 128)
        go(moe_plan_kernel<2, kBf16, true>);
    else if (E <= 256)
        go(moe_plan_kernel<4, kBf16, true>);
    else
        go(moe_plan_kernel<16, kBf16, true>);
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
    int *plan = static_cast<int *>(ws);
    const int records = (int)moe_plan_records(w.E, P);
    uint16_t *hidden = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(ws) + moe_plan_bytes(w.E, P));
    if (r.bf16)
        launch_plan<true>(r, T, w.E, plan, s);
    else
        launch_plan<false>(r, T, w.E, plan, s);
    const int units = records * (w.I / 64);  // runs of four tiles, rounded up to whole rounds of the XCDs
    const int blocks = (units + kXcds - 1) / kXcds * kXcds * 4;
    hipLaunchKernelGGL(moe_up_kernel, dim3(blocks), dim3(kUpWaves * kWave), 0, s, x, ldx, r.k, w.w1, w.s1, w.z1, w.H,
                       w.I, plan, records, hidden);
    const int slots = P * kDownWaves < kMoePairs ? P * kDownWaves : kMoePairs;
    hipLaunchKernelGGL(moe_down_kernel, dim3(w.H / 16), dim3(kDownWaves * kWave), slots * 64, s, hidden, w.w2, w.s2,
                       w.z2, w.H, w.I, T, r.k, w.E, plan, records, r.ids, r.weights, out, ldo);
    return (int)hipGetLastError();
}

}  // namespace ck
