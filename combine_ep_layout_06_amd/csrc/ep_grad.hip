// The gradients that are bound by their bytes, on gfx950: combine's, and those of a dense product's
// activation and bias.
#include "ep_product.h"

#include <algorithm>

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

__device__ __forceinline__ u32x4 pack8(const float (&v)[8])
{
    u32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = bf16_rne(v[2 * i]) | (bf16_rne(v[2 * i + 1]) << 16);
    return d;
}

// Combine's gradient: out[t] = sum_j w[t][j] y[row(t, j)] gives
//   dy[row] = bf16(w[t][j] * dout[t]),  dw[t][j] = sum_h dout[t][h] y[row][h]
// W wavefronts per pair: one where there are pairs enough for every CU, else the workgroup's four
// (129 tokens, top-8, H = 2056: 10.9 -> 10.1 us with the launch). A lane has kChunks 16-byte chunks of
// both rows in flight (one: 57 us). 4096 tokens, top-8, H = 2048: 49 us, bound by its bytes (268 MB, half
// of them written: 5.6 TB/s, a copy has 4.7).
constexpr int kChunks = 4;
constexpr int kManyPairs = 8192;   // 8 wavefronts for each SIMD
constexpr int64_t kMostGroups = 1 << 23;       // of a row of the grid, which holds fewer than 2^32 threads

template <int W>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(
    const u32x4 *__restrict__ dout, const u32x4 *y, const int32_t *__restrict__ idx,
    const int32_t *__restrict__ slot, const float *__restrict__ topk_w, u32x4 *dy,
    float *__restrict__ dw, int pairs, int H8, int E, int C, int K, const int32_t *__restrict__ poff,
    int prows)
{
    __shared__ float sums[kWaves];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kWaves / W) + wave / W;
    if (i >= pairs) return;                    // W > 1: the whole workgroup
    const int row = __builtin_amdgcn_readfirstlane(pair_row(idx[i], slot[i], E, C, poff, prows));
    if (row < 0) {
        if (wave % W == 0 && lane == 0) dw[i] = 0.0f;
        return;
    }
    const float w = topk_w[i];
    const u32x4 *d = dout + (size_t)(i / K) * H8, *yr = y + (size_t)row * H8;
    u32x4 *o = dy + (size_t)row * H8;
    float sum = 0.0f;
    for (int c0 = wave % W * kWave + lane; c0 < H8; c0 += kChunks * W * kWave) {
        u32x4 a[kChunks], b[kChunks];
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {    // beyond the row: its last chunk again
            const int c = min(c0 + u * W * kWave, H8 - 1);
            a[u] = d[c];
            b[u] = load16<true>(yr + c);
        }
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int c = c0 + u * W * kWave;
            if (c >= H8) break;
            float g[8], v[8];
            unpack8(a[u], g);
            unpack8(b[u], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum = __builtin_fmaf(g[k], v[k], sum);
                g[k] *= w;
            }
            store16<true>(o + c, pack8(g));
        }
    }
#pragma unroll
    for (int x = 1; x < kWave; x *= 2) sum += __shfl_xor(sum, x);
    if constexpr (W > 1) {
        if (lane == 0) sums[wave] = sum;
        __syncthreads();
        sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    }
    if (wave % W == 0 && lane == 0) dw[i] = sum;
}

// dz = bf16(dout * act'(z)) and, per kGradRows rows, the columns' sums of the unrounded dz: bound by its
// bytes, kGradAtOnce rows of both in flight. 4096 x 4096, silu: 256 threads 31 us, 512 28 (3.6 TB/s). dz is
// rounded because it is the matrix instruction's operand twice: dx and dw are then 0.0023 of their norm from
// the values in 64 bits, where their own rounding to bf16 makes 0.0017 (without an activation and with relu dz
// is exact, and they are too). dz in two parts of bf16 would make it 0.0017 for twice the products, which are
// 153 of the 185 us of 4096 rows x 2048 x 4096.
constexpr int kGradRows = kLinearGradRows;
constexpr int kGradThreads = 512, kGradWaves = kGradThreads / kWave;
constexpr int kGradAtOnce = 4;     // rows of a wavefront in flight

__global__ __launch_bounds__(kGradThreads) void act_grad_kernel(
    const uint16_t *__restrict__ dout, const uint16_t *__restrict__ z, uint16_t *__restrict__ dz,
    float *__restrict__ part, int T, int N, int act)
{
    __shared__ float sums[kGradWaves][kWave][9];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int c = (blockIdx.x * kWave + lane) * 8;
    float sum[8] = {};
    if (c < N) {
        const int first = blockIdx.y * kGradRows + wave, end = min((int)(blockIdx.y + 1) * kGradRows, T);
        for (int t0 = first; t0 < end; t0 += kGradAtOnce * kGradWaves) {
            u32x4 d[kGradAtOnce], v[kGradAtOnce];
#pragma unroll
            for (int i = 0; i < kGradAtOnce; ++i) {    // a row that is not there: the last one again
                const size_t at = (size_t)min(t0 + i * kGradWaves, end - 1) * N + c;
                d[i] = *reinterpret_cast<const u32x4 *>(dout + at);
                if (act != EP_ACT_NONE) v[i] = *reinterpret_cast<const u32x4 *>(z + at);
            }
#pragma unroll
            for (int i = 0; i < kGradAtOnce; ++i) {
                const int t = t0 + i * kGradWaves;
                if (t >= end) break;
                float g[8];
                unpack8(d[i], g);
                if (act != EP_ACT_NONE) {
                    float a[8];
                    unpack8(v[i], a);
#pragma unroll
                    for (int k = 0; k < 8; ++k) g[k] *= act_grad(act, a[k]);
                    *reinterpret_cast<u32x4 *>(dz + (size_t)t * N + c) = pack8(g);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += g[k];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[wave][lane][k] = sum[k];
    __syncthreads();
    for (int i = threadIdx.x; i < kWave * 8; i += kGradThreads) {
        const int col = blockIdx.x * kWave * 8 + i;
        if (col < N) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kGradWaves; ++w) s += sums[w][i >> 3][i & 7];
            part[(size_t)blockIdx.y * N + col] = s;
        }
    }
}

// The sums of the workgroups' sums: 64 columns a workgroup, a quarter of the rows a wavefront (a column's
// sums one after the other in one lane took 20 us for 4096 x 4096, this 5).
__global__ __launch_bounds__(kThreads) void bias_grad_kernel(const float *__restrict__ part,
                                                             float *__restrict__ dbias, int chunks, int N)
{
    __shared__ float sums[kWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int c = blockIdx.x * kWave + lane;
    float s = 0.0f;
    if (c < N) {
#pragma unroll 8
        for (int i = wave; i < chunks; i += kWaves) s += part[(size_t)i * N + c];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < N) dbias[c] = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
}

}  // namespace

hipError_t launch_combine_grad(const ep_shape_t &s, const uint16_t *dout, const uint16_t *y,
                               const int32_t *idx, const int32_t *slot, const float *w, uint16_t *dy,
                               float *dw, hipStream_t stream, RowMap map)
{
    const int pairs = s.T * s.K;
    if (pairs == 0) return hipSuccess;
    auto go = [&](auto kernel, int per) {
        const int64_t groups = ((int64_t)pairs + per - 1) / per;
        const dim3 grid((unsigned)std::min(groups, kMostGroups), (unsigned)((groups + kMostGroups - 1) / kMostGroups));
        return launch(kernel, grid, dim3(kThreads), 0, stream, reinterpret_cast<const u32x4 *>(dout),
                      reinterpret_cast<const u32x4 *>(y), idx, slot, w, reinterpret_cast<u32x4 *>(dy), dw, pairs,
                      s.H / 8, s.E, s.C, s.K, map.offset, map.rows);
    };
    return pairs >= kManyPairs ? go(combine_grad_kernel<1>, kWaves) : go(combine_grad_kernel<kWaves>, 1);
}

hipError_t launch_act_grad(const uint16_t *dout, const uint16_t *z, uint16_t *dz, float *part,
                           float *dbias, int T, int N, int act, hipStream_t stream)
{
    const int chunks = (T + kGradRows - 1) / kGradRows;
    if (chunks > 0) {
        const hipError_t e = launch(act_grad_kernel, dim3((N / 8 + kWave - 1) / kWave, chunks),
                                    dim3(kGradThreads), 0, stream, dout, z, dz, part, T, N, act);
        if (e != hipSuccess) return e;
    }
    return launch(bias_grad_kernel, dim3((N + kWave - 1) / kWave), dim3(kThreads), 0, stream, part, dbias,
                  chunks, N);
}

}  // namespace ep
