// Low-rank adapters of many requests beside a shared projection:
//   out[m] = base[m] + scaling[a] B_a (A_a x_m),  a = index[m] (outside [0, L): base[m]).
//
// Two launches.  The first forms v = A_a x_m (fp32, in parts of the K columns so
// that few rows still fill the chip), the second adds B_a v to base.  Rows of
// one adapter share its weights: the 64 lanes of a wave read the indices of a
// window of rows, a ballot gives the rows of one adapter, and those rows
// (wherever they lie in the window) fill the 16-row tiles of the bf16 MFMA.
//   * up to kPerRowMax rows (decode), a workgroup is started for every row and
//     the first row of each adapter in the window does the work for all of
//     them: requests of unlike adapters run side by side;
//   * above (prompts, where neighbours share an adapter), a workgroup
//     takes a window and goes through its adapters one after the other.
// v enters the second product as two bf16 (16 significant bits) side by side in
// the MFMA's 32 columns of k: columns 0-15 the first parts, 16-31 the second,
// both against the same 16 columns of B_a.
// The work is bound by memory: x, base and out once, the used adapters once.
#include "rows_device.h"
#include "rows_launch.h"

namespace ck {
namespace {

constexpr int64_t kPerRowMax = kLoraPerRowMax;
constexpr int kRankBlock = kLoraRankBlock;  // ranks per workgroup (first product) or pass (second)

// The rows of a window of kWin, and those that share one adapter.
struct RowSet {
    int order;  // lane i: the i-th row of the set (window-relative)
    int count;
};
__device__ __forceinline__ int window_adapter(const int32_t *index, int64_t M, int64_t L, int64_t row0, int win,
                                              int lane)
{
    if (lane >= win || row0 + lane >= M)
        return -2;
    const int a = index[row0 + lane];
    return a < 0 || a >= L ? -1 : a;
}
__device__ __forceinline__ RowSet row_set(uint64_t mask, int lane)
{
    const uint64_t below = (uint64_t(1) << lane) - 1;
    const int count = __builtin_popcountll(mask);
    const int pos = (mask >> lane) & 1 ? __builtin_popcountll(mask & below)
                                       : count + __builtin_popcountll(~mask & below);
    return RowSet{__builtin_amdgcn_ds_permute(4 * pos, lane), count};
}

// Calls f(adapter, rows) for each adapter of the window, or, per row, for the
// adapter whose first row this workgroup was started for.
template <bool kPerRow, class F>
__device__ __forceinline__ void for_adapters(int mine, int me, int lane, F &&f)
{
    uint64_t left = __ballot(mine != -2);
    if constexpr (kPerRow) {
        const int a = __builtin_amdgcn_readlane(mine, me);
        const uint64_t mask = __ballot(mine == a);
        if (__builtin_ctzll(mask) == me)
            f(a, row_set(mask, lane));
    } else {
        while (left) {
            const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
            const uint64_t mask = __ballot(mine == a);
            left &= ~mask;
            f(a, row_set(mask, lane));
        }
    }
}

__device__ __forceinline__ int adapter_rank(const int32_t *ranks, int a, int R)
{
    return ranks ? min(max(ranks[a], 0), R) : R;
}

// First product.  Grid: (rows or windows, parts of K, blocks of 64 ranks); the
// workgroup's waves split its part of K and are summed through LDS.
template <bool kPerRow, int kWaves, int kTiles>
__global__ __launch_bounds__(kWaves * kWave) void lora_shrink_kernel(
    const uint16_t *__restrict__ x, int64_t M, int K, int64_t ldx, const int32_t *__restrict__ index, int64_t L,
    int R, const uint16_t *__restrict__ a_w, const int32_t *__restrict__ ranks, float *__restrict__ v)
{
    constexpr int kWin = kPerRow ? kLoraWindow : 16 * kTiles;
    constexpr int kRT = kRankBlock / 16;
    __shared__ float s_red[kWaves][kTiles][kRT][256];
    __shared__ int s_rows[kWave];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int l16 = lane % 16, quarter = lane / 16;
    const int64_t row0 = kPerRow ? (int64_t)blockIdx.x / kWin * kWin : (int64_t)blockIdx.x * kWin;
    const int rb = blockIdx.z * kRankBlock;
    const int KG = K / 64, parts = gridDim.y * kWaves, part = blockIdx.y * kWaves + wave;
    const int g0 = (int)((int64_t)part * KG / parts), g1 = (int)((int64_t)(part + 1) * KG / parts);
    const int mine = window_adapter(index, M, L, row0, kWin, lane);

    for_adapters<kPerRow>(mine, (int)(blockIdx.x % kWin), lane, [&](int ad, RowSet rows) {
        if (ad < 0)
            return;
        const int rank = adapter_rank(ranks, ad, R);
        if (rank <= rb)
            return;
        const int nrt = min(kRT, (rank - rb + 15) / 16);
        const uint16_t *arow[kRT];
#pragma unroll
        for (int rt = 0; rt < kRT; ++rt)
            arow[rt] = a_w + ((int64_t)ad * R + min(rb + 16 * rt + l16, rank - 1)) * K + 16 * quarter;
        for (int p0 = 0; p0 < rows.count; p0 += 16 * kTiles) {
            const uint16_t *xrow[kTiles];
#pragma unroll
            for (int mt = 0; mt < kTiles; ++mt)
                xrow[mt] = x + (row0 + __shfl(rows.order, min(p0 + 16 * mt + l16, rows.count - 1))) * ldx + 16 * quarter;
            v4f acc[kTiles][kRT];
#pragma unroll
            for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                for (int rt = 0; rt < kRT; ++rt)
                    acc[mt][rt] = v4f{0.f, 0.f, 0.f, 0.f};
            for (int g = g0; g < g1; ++g) {
                v8bf xv[kTiles][2];
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        xv[mt][h] = __builtin_bit_cast(
                            v8bf, *reinterpret_cast<const u32x4 *>(xrow[mt] + g * 64 + 8 * h));
#pragma unroll
                for (int rt = 0; rt < kRT; ++rt) {
                    if (rt < nrt) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const v8bf av = __builtin_bit_cast(
                                v8bf, *reinterpret_cast<const u32x4 *>(arow[rt] + g * 64 + 8 * h));
#pragma unroll
                            for (int mt = 0; mt < kTiles; ++mt)
                                acc[mt][rt] = mfma16(xv[mt][h], av, acc[mt][rt]);
                        }
                    }
                }
            }
            __syncthreads();  // the previous tile's sums and rows have been read
            if (wave == 0)
                s_rows[lane] = rows.order;
#pragma unroll
            for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                for (int rt = 0; rt < kRT; ++rt)
                    if (rt < nrt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s_red[wave][mt][rt][i * kWave + lane] = acc[mt][rt][i];
            __syncthreads();
            // Threads in the order (tile, row, rank tile, rank): 16-rank runs.
            for (int o = threadIdx.x; o < kTiles * 16 * nrt * 16; o += kWaves * kWave) {
                const int r = o % 16, rt = o / 16 % nrt, row = o / (16 * nrt) % 16, mt = o / (256 * nrt);
                const int p = p0 + 16 * mt + row;
                if (p < rows.count && rb + 16 * rt + r < rank) {
                    const int at = (row % 4) * kWave + (row / 4) * 16 + r;
                    float t = s_red[0][mt][rt][at];
#pragma unroll
                    for (int w = 1; w < kWaves; ++w)
                        t += s_red[w][mt][rt][at];
                    v[((int64_t)blockIdx.y * M + row0 + s_rows[p]) * R + rb + 16 * rt + r] = t;
                }
            }
        }
    });
}

// The 8 ranks from r on of one row's v: parts summed in order, scaled, 0 from
// `rank` on; the first or the second bf16 of each.
__device__ __forceinline__ v8bf load_v8(const float *vrow, int64_t part_stride, int parts, int r, int rank,
                                        float scale, bool second)
{
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        t[e] = 0.f;
    if (r < rank) {  // v is written up to rank; the rest of its 8 are not used
        for (int s = 0; s < parts; ++s) {
            const float *p = vrow + s * part_stride + r;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const v4f u = *reinterpret_cast<const v4f *>(p + 4 * q);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    t[4 * q + e] += u[e];
            }
        }
    }
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint16_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            split_bf16(r + 2 * q + e < rank ? scale * t[2 * q + e] : 0.f, hi[e], lo[e]);
        w[q] = second ? lo[0] | (uint32_t)lo[1] << 16 : hi[0] | (uint32_t)hi[1] << 16;
    }
    return __builtin_bit_cast(v8bf, w);
}

// The 8 ranks from r on of one row of B_a, 0 from `rank` on (whatever is stored there).
__device__ __forceinline__ v8bf load_b8(const uint16_t *brow, int r, int rank)
{
    u32x4 w = {0u, 0u, 0u, 0u};
    if (r < rank)
        w = *reinterpret_cast<const u32x4 *>(brow + r);
    if (r + 8 > rank)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] &= (r + 2 * q < rank ? 0xffffu : 0u) | (r + 2 * q + 1 < rank ? 0xffff0000u : 0u);
    return __builtin_bit_cast(v8bf, w);
}

// Second product.  Grid: rows or windows, by columns / (32 kWaves kCols).  A wave
// owns kCols tiles of 32 columns of the output; two MFMA tiles with interleaved
// columns leave each lane 8 consecutive ones of its row, one 16-byte store.
template <bool kPerRow, int kWaves, int kTiles, int kCols>
__global__ __launch_bounds__(kWaves * kWave) void lora_expand_kernel(
    const float *__restrict__ v, int parts, int64_t M, const int32_t *__restrict__ index, int64_t L, int R,
    const uint16_t *__restrict__ b_w, const float *__restrict__ scaling, const int32_t *__restrict__ ranks, int N,
    const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo)
{
    constexpr int kSteps = kRankBlock / 16;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int l16 = lane % 16, quarter = lane / 16;
    const int ctiles = (N + 32 * kWaves * kCols - 1) / (32 * kWaves * kCols);
    const int unit = blockIdx.x / ctiles;
    const int64_t row0 = (int64_t)(kPerRow ? unit / kLoraWindow : unit) * kLoraWindow;
    const int c0 = (blockIdx.x % ctiles * kWaves + wave) * 32 * kCols;
    const int mine = window_adapter(index, M, L, row0, kLoraWindow, lane);

    for_adapters<kPerRow>(mine, unit % kLoraWindow, lane, [&](int ad, RowSet rows) {
        const int rank = ad < 0 ? 0 : adapter_rank(ranks, ad, R);
        const float scale = ad >= 0 && scaling ? scaling[ad] : 1.f;
        const int passes = max(1, (rank + kRankBlock - 1) / kRankBlock);
        for (int p0 = 0; p0 < rows.count; p0 += 16 * kTiles) {
            int64_t row[kTiles];
            v8bf vf[kTiles][kSteps];
#pragma unroll
            for (int mt = 0; mt < kTiles; ++mt)
                row[mt] = row0 + __shfl(rows.order, min(p0 + 16 * mt + l16, rows.count - 1));
            for (int ct = 0; ct < kCols; ++ct) {
                const int n = c0 + 32 * ct + 8 * quarter;
                if (c0 + 32 * ct >= N)
                    break;
                u32x4 bv[kTiles];
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt)
                    bv[mt] = base && n < N ? *reinterpret_cast<const u32x4 *>(base + row[mt] * ldb + n)
                                           : u32x4{0u, 0u, 0u, 0u};
                v4f acc[kTiles][2];
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt)
                    acc[mt][0] = acc[mt][1] = v4f{0.f, 0.f, 0.f, 0.f};
                for (int pass = 0; pass < passes; ++pass) {
                    const int r0 = pass * kRankBlock + 8 * (quarter % 2);
                    if (ct == 0 || passes > 1) {
#pragma unroll
                        for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                            for (int st = 0; st < kSteps; ++st)
                                if (pass * kRankBlock + 16 * st < rank)
                                    vf[mt][st] = load_v8(v + row[mt] * R, M * R, parts, r0 + 16 * st, rank, scale,
                                                         quarter >= 2);
                    }
#pragma unroll
                    for (int st = 0; st < kSteps; ++st) {
                        if (pass * kRankBlock + 16 * st < rank) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int nb = min(c0 + 32 * ct + 8 * (l16 / 4) + 4 * h + l16 % 4, N - 1);
                                const v8bf bf = load_b8(b_w + ((int64_t)ad * N + nb) * R, r0 + 16 * st, rank);
#pragma unroll
                                for (int mt = 0; mt < kTiles; ++mt)
                                    acc[mt][h] = mfma16(bf, vf[mt][st], acc[mt][h]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt) {
                    if (p0 + 16 * mt + l16 < rows.count && n < N) {
                        u32x4 o;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const v4f &t = acc[mt][q / 2];
                            o[q] = pack_bf16x2(t[2 * q % 4] + bf16_to_f32(bv[mt][q] & 0xffffu),
                                               t[2 * q % 4 + 1] + __uint_as_float(bv[mt][q] & 0xffff0000u));
                        }
                        *reinterpret_cast<u32x4 *>(out + row[mt] * ldo + n) = o;
                    }
                }
            }
        }
    });
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
    const int parts = lora_splits(M, K, R, L);
    const unsigned rb = (unsigned)lora_ceil(R, kRankBlock);
    if (M <= kPerRowMax) {
        hipLaunchKernelGGL((lora_shrink_kernel<true, 4, 1>), dim3((unsigned)M, parts, rb), dim3(4 * kWave), 0, s, x, M,
                           K, ldx, index, L, R, a, ranks, ws);
        hipLaunchKernelGGL((lora_expand_kernel<true, 4, 1, 1>), dim3((unsigned)(lora_ceil(N, 128) * M)),
                           dim3(4 * kWave), 0, s, ws, parts, M, index, L, R, b, scaling, ranks, N, base, ldb, out, ldo);
    } else {
        hipLaunchKernelGGL((lora_shrink_kernel<false, 8, 2>), dim3((unsigned)lora_ceil(M, 32), parts, rb),
                           dim3(8 * kWave), 0, s, x, M, K, ldx, index, L, R, a, ranks, ws);
        hipLaunchKernelGGL((lora_expand_kernel<false, 4, 4, 2>),
                           dim3((unsigned)(lora_ceil(N, 256) * lora_ceil(M, kLoraWindow))), dim3(4 * kWave), 0, s,
                           ws, parts, M, index, L, R, b, scaling, ranks, N, base, ldb, out, ldo);
    }
    return (int)hipGetLastError();
}

}  // namespace ck
