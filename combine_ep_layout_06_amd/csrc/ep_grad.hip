// The gradients that are bound by their bytes, on gfx950: combine's, and those of a dense product's
// activation and bias.
#include "ep_product.h"

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
// One wavefront per pair.
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(
    const u32x4 *__restrict__ dout, const u32x4 *__restrict__ y, const int32_t *__restrict__ idx,
    const int32_t *__restrict__ slot, const float *__restrict__ topk_w, u32x4 *__restrict__ dy,
    float *__restrict__ dw, int pairs, int H8, int E, int C, int K, const int32_t *__restrict__ poff,
    int prows)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int i = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (i >= pairs) return;
    const int row = __builtin_amdgcn_readfirstlane(pair_row(idx[i], slot[i], E, C, poff, prows));
    if (row < 0) {
        if (lane == 0) dw[i] = 0.0f;
        return;
    }
    const float w = topk_w[i];
    const u32x4 *d = dout + (size_t)(i / K) * H8, *yr = y + (size_t)row * H8;
    u32x4 *o = dy + (size_t)row * H8;
    float sum = 0.0f;
    for (int c = lane; c < H8; c += kWave) {
        float a[8], b[8];
        unpack8(d[c], a);
        unpack8(yr[c], b);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sum = __builtin_fmaf(a[k], b[k], sum);
            a[k] *= w;
        }
        o[c] = pack8(a);
    }
#pragma unroll
    for (int x = 1; x < kWave; x *= 2) sum += __shfl_xor(sum, x);
    if (lane == 0) dw[i] = sum;
}

// dz = bf16(dout * act'(z)) and, per kGradRows rows, the columns' sums of the unrounded dz.
constexpr int kGradRows = kLinearGradRows;
constexpr int kGradAtOnce = 4;     // rows of a wavefront in flight

__global__ __launch_bounds__(kThreads) void act_grad_kernel(
    const uint16_t *__restrict__ dout, const uint16_t *__restrict__ z, uint16_t *__restrict__ dz,
    float *__restrict__ part, int T, int N, int act)
{
    __shared__ float sums[kWaves][kWave][9];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int c = (blockIdx.x * kWave + lane) * 8;
    float sum[8] = {};
    if (c < N) {
        const int first = blockIdx.y * kGradRows + wave, end = min((int)(blockIdx.y + 1) * kGradRows, T);
        for (int t0 = first; t0 < end; t0 += kGradAtOnce * kWaves) {
            u32x4 d[kGradAtOnce], v[kGradAtOnce];
#pragma unroll
            for (int i = 0; i < kGradAtOnce; ++i) {    // a row that is not there: the last one again
                const size_t at = (size_t)min(t0 + i * kWaves, end - 1) * N + c;
                d[i] = *reinterpret_cast<const u32x4 *>(dout + at);
                if (act != EP_ACT_NONE) v[i] = *reinterpret_cast<const u32x4 *>(z + at);
            }
#pragma unroll
            for (int i = 0; i < kGradAtOnce; ++i) {
                const int t = t0 + i * kWaves;
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
    for (int i = threadIdx.x; i < kWave * 8; i += kThreads) {
        const int col = blockIdx.x * kWave * 8 + i;
        if (col < N) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) s += sums[w][i >> 3][i & 7];
            part[(size_t)blockIdx.y * N + col] = s;
        }
    }
}

// The sums of the workgroups' sums: 64 columns a workgroup, a quarter of the rows a wavefront.
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
    return launch(combine_grad_kernel, dim3((pairs + (kWaves - 1)) / kWaves), dim3(kThreads), 0, stream,
                  reinterpret_cast<const u32x4 *>(dout), reinterpret_cast<const u32x4 *>(y), idx, slot, w,
                  reinterpret_cast<u32x4 *>(dy), dw, pairs, s.H / 8, s.E, s.C, s.K, map.offset, map.rows);
}

hipError_t launch_act_grad(const uint16_t *dout, const uint16_t *z, uint16_t *dz, float *part,
                           float *dbias, int T, int N, int act, hipStream_t stream)
{
    const int chunks = (T + kGradRows - 1) / kGradRows;
    if (chunks > 0) {
        const hipError_t e = launch(act_grad_kernel, dim3((N / 8 + kWave - 1) / kWave, chunks),
                                    dim3(kThreads), 0, stream, dout, z, dz, part, T, N, act);
        if (e != hipSuccess) return e;
    }
    return launch(bias_grad_kernel, dim3((N + kWave - 1) / kWave), dim3(kThreads), 0, stream, part, dbias,
                  chunks, N);
}

}  // namespace ep
