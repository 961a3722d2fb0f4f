// The gradients that are bound by their bytes, on gfx950: combine's, and those of a dense product's
// activation and bias.
#include "ep_product.h"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

__device__ __forceinline__ void unpack8(u32x4 d, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(d[i]);
        v[2 * i + 1] = bf16_hi(d[i]);
    }
}

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

__device__ __forceinline__ float act_grad(int act, float z)
{
    if (act == EP_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == EP_ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(__builtin_fmaf(__expf(-z), 0x1p-4f, 0x1p-4f)) * 0x1p-4f;
        return s * __builtin_fmaf(z, 1.0f - s, 1.0f);
    }
    // Phi(z) + z phi(z)
    return __builtin_fmaf(0.5f, erff(z * 0.70710678f), 0.5f) + z * __expf(-0.5f * z * z) * 0.39894228f;
}

__global__ __launch_bounds__(kThreads) void act_grad_kernel(
    const uint16_t *__restrict__ dout, const uint16_t *__restrict__ z, uint16_t *__restrict__ dz,
    float *__restrict__ part, int T, int N, int act)
{
    __shared__ float sums[kWaves][kWave][9];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int c = (blockIdx.x * kWave + lane) * 8;
    float sum[8] = {};
    if (c < N) {
        const int end = min((int)(blockIdx.y + 1) * kGradRows, T);
        for (int t = blockIdx.y * kGradRows + wave; t < end; t += kWaves) {
            const size_t at = (size_t)t * N + c;
            float d[8];
            unpack8(*reinterpret_cast<const u32x4 *>(dout + at), d);
            if (act != EP_ACT_NONE) {
                float v[8];
                unpack8(*reinterpret_cast<const u32x4 *>(z + at), v);
#pragma unroll
                for (int k = 0; k < 8; ++k) d[k] *= act_grad(act, v[k]);
                *reinterpret_cast<u32x4 *>(dz + at) = pack8(d);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += d[k];
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

__global__ __launch_bounds__(kThreads) void bias_grad_kernel(const float *__restrict__ part,
                                                             float *__restrict__ dbias, int chunks, int N)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= N) return;
    float s = 0.0f;
    for (int i = 0; i < chunks; ++i) s += part[(size_t)i * N + c];
    dbias[c] = s;
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
    return launch(bias_grad_kernel, dim3((N + kThreads - 1) / kThreads), dim3(kThreads), 0, stream, part,
                  dbias, chunks, N);
}

}  // namespace ep
