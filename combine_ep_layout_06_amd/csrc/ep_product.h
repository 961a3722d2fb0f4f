// The bf16 products: host launchers (internal header).
#pragma once

#include "ep_expert.h"

namespace ep {

// One bf16 product over the rows of E experts (padded [E][C], packed with `offset`, or, with count
// null, the C rows of a dense matrix, E = 1).
//
//   forward   out[r][c] = sum_k x[r][k] w[e][c][k]    w [E][n][k]
//   dgrad     out[r][c] = sum_k x[r][k] w[e][k][c]    w [E][k][n]
//   wgrad     out[e][r][c] = sum_i x[i][r] w[i][c]    x [rows][m], w [rows][n], i over e's rows
struct Product {
    const uint16_t *x, *w;
    const int32_t *count;     // [E] rows per expert; null: dense
    const int32_t *offset;    // packed: first row of each expert; null: padded
    int E, C, rows;
    int k;                    // length of the sums (wgrad: not used)
    int m;                    // wgrad: rows of an output matrix
    int n;                    // columns of the output (SwiGLU: 2I)
    int pairs;                // rows laid out: chooses the grid, nothing else
    // the epilogue
    void *out;                // bf16; fp32 for the fp32 weight gradient
    uint16_t *out2;           // SwiGLU: gu or null; linear: z or null
    const uint16_t *in;       // SwiGLU gradient: gu; linear: residual or null
    const uint16_t *bias;     // linear: [n] or null
    int act;                  // linear: EP_ACT_*
    int accumulate;           // fp32 weight gradient: add to what is there
};

hipError_t launch_expert_gemm(const Product &p, hipStream_t stream);
hipError_t launch_expert_swiglu(const Product &p, hipStream_t stream);
hipError_t launch_expert_dgrad(const Product &p, hipStream_t stream);
hipError_t launch_expert_swiglu_dgrad(const Product &p, hipStream_t stream);
hipError_t launch_expert_wgrad(const Product &p, bool f32, hipStream_t stream);
hipError_t launch_linear(const Product &p, hipStream_t stream);

// The products for few rows, and whether they are the better ones for these rows (some; of a packed
// buffer with some).
bool few_rows(const Product &p, bool swiglu);
hipError_t launch_few_gemm(const Product &p, hipStream_t stream);
hipError_t launch_few_swiglu(const Product &p, hipStream_t stream);
hipError_t launch_few_linear(const Product &p, hipStream_t stream);
bool few_dgrad(const Product &p);
hipError_t launch_few_dgrad(const Product &p, bool swiglu, hipStream_t stream);
// And whether a weights' gradient is one of few tiles and long sums.
bool few_wgrad(const Product &p);
hipError_t launch_few_wgrad(const Product &p, bool f32, hipStream_t stream);

hipError_t launch_combine_grad(const ep_shape_t &s, const uint16_t *dout, const uint16_t *y,
                               const int32_t *idx, const int32_t *slot, const float *w, uint16_t *dy,
                               float *dw, hipStream_t stream, RowMap map = RowMap());

// Rows whose columns' sums a workgroup of the activation's gradient takes; grid.y holds 65535 of them.
constexpr int kLinearGradRows = 64;

// dz = bf16(dout * act'(z)) (not written without an activation) and dbias, the columns' sums of the
// unrounded dz, through `part`: ceil(T / kLinearGradRows) rows of N.
hipError_t launch_act_grad(const uint16_t *dout, const uint16_t *z, uint16_t *dz, float *part,
                           float *dbias, int T, int N, int act, hipStream_t stream);

#if defined(__HIPCC__)

#if defined(__HIP_DEVICE_COMPILE__)
// The kernel's argument, a Product, read anew: what only the epilogue uses takes no register through the products.
__device__ __forceinline__ const __attribute__((address_space(4))) Product &argument()
{
    const auto at = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
    uint32_t lo, hi;
    asm volatile("" : "=s"(lo) : "0"(__builtin_amdgcn_readfirstlane((int)(uint32_t)at)));
    asm volatile("" : "=s"(hi) : "0"(__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32))));
    return *reinterpret_cast<const __attribute__((address_space(4))) Product *>((uint64_t)hi << 32 | lo);
}

// The lane, counted anew: what is computed from it is worked out where it is used, and takes no
// register through the products (which need them all).
__device__ __forceinline__ int lane_now()
{
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
    return l;
}

// A lane's byte offset past every buffer's end: nothing is stored there, and loads give 0.
constexpr uint32_t kNone = 0x80000000u;

typedef __attribute__((address_space(3))) uint8_t *LdsBytes;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 *LdsTr;
typedef __attribute__((address_space(3))) bf16x8 *LdsRows;

// A buffer's descriptor, of `bytes` from p: loads past them give 0.
__device__ __forceinline__ i32x4 buffer(const void *p, int64_t bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const int n = bytes <= 0 ? 0 : bytes > 0x7FFFFFFF ? 0x7FFFFFFF : (int)bytes;
    return i32x4{(int)(uint32_t)a, (int)(uint32_t)(a >> 32), n, 0x00027000};
}

// 16 bytes a lane from buffer `b` to 1 KiB of LDS from `to` on, lane after lane. Written out, because
// the compiler cannot tell which of the stages a load of the builtin's form fills once paths meet, and
// then waits for all of them before the next LDS read. It has no register output: the waits for it are
// the kernels' own, and the compiler's own waits for later loads are only stricter by it. Nothing
// else in these kernels uses m0.
__device__ __forceinline__ void load_lds(i32x4 b, uint8_t *to, uint32_t off, uint32_t soff)
{
    const uint32_t at = (uint32_t)(uintptr_t)(LdsBytes)to;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(uniform(at)), "v"(off),
                    "s"(i32x4{uniform(b[0]), uniform(b[1]), uniform(b[2]), uniform(b[3])}),
                    "s"(uniform(soff)) : "memory");
}

// Four consecutive sum indexes of one column from LDS: lane i of 16 gives the address of columns (i & 3) *
// 4 .. of sum index i >> 2, and receives column i.
__device__ __forceinline__ bf16x8 read_transposed(uint32_t at, uint32_t second)
{
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr)(uintptr_t)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr)(uintptr_t)second);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
#endif

__device__ __forceinline__ void unpack8(u32x4 d, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(d[i]);
        v[2 * i + 1] = bf16_hi(d[i]);
    }
}

// 1 / (1 + exp(-g)), the reciprocal as in swiglu().
__device__ __forceinline__ float sigmoid(float g)
{
    return __builtin_amdgcn_rcpf(__builtin_fmaf(__expf(-g), 0x1p-4f, 0x1p-4f)) * 0x1p-4f;
}

// A constant put into a register where it is used, and not kept in one through a kernel's loops.
#define EP_HERE(value)                                                                          \
    [] {                                                                                        \
        float r;                                                                                \
        asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "i"(__builtin_bit_cast(int, value)));        \
        return r;                                                                               \
    }()

// The normal distribution Phi(z) and, in `density`, exp(-z^2 / 2). With x = |z| / sqrt(2) and t = 1 / (1 +
// 0.41 x) the tail beyond |z| is erfc(x) / 2 = exp(-x^2) t q(t). q is fitted to it for x up to 9.6 with an
// error of 2.3e-7 (1 + 8 x^2) of the tail at most: near 0, where it shows beside 1, the least, and far out a few
// times what the rounding of exp's argument makes. So the tail keeps its relative accuracy, which a value of z
// far below 0 needs: with fp32's roundings Phi is within 2^-21, and for z < 0 within
// (1 + z^2) 2^-19 of its own size down to z = -13.1 (below it the tail ends as a zero).
__device__ __forceinline__ float normal_cdf(float z, float &density)
{
    const float x = __builtin_fabsf(z) * 0.70710678f;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(EP_HERE(0.41f), x, 1.0f));
    float y = __builtin_fmaf(EP_HERE(-0.0889302567f), t, EP_HERE(0.28596624732f));
    y = __builtin_fmaf(y, t, EP_HERE(-0.0951913446f));
    y = __builtin_fmaf(y, t, EP_HERE(0.1812158674f));
    y = __builtin_fmaf(y, t, EP_HERE(0.1000034884f));
    y = __builtin_fmaf(y, t, EP_HERE(0.1169361025f));
    density = __expf(-x * x);
    y *= t * density;
    return z < 0.0f ? y : 1.0f - y;
}

__device__ __forceinline__ float activate(int act, float z)
{
    float density;
    if (act == EP_ACT_RELU) return z > 0.0f || z != z ? z : 0.0f;
    if (act == EP_ACT_SILU) return z * sigmoid(z);
    if (act == EP_ACT_GELU) return z * normal_cdf(z, density);
    return z;
}

// The derivative of activate().
__device__ __forceinline__ float act_grad(int act, float z)
{
    if (act == EP_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == EP_ACT_SILU) {
        const float s = sigmoid(z);
        return s * __builtin_fmaf(z, 1.0f - s, 1.0f);
    }
    float density;                             // Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi)
    const float cdf = normal_cdf(z, density);
    return __builtin_fmaf(z * 0.39894228f, density, cdf);
}

#endif

}  // namespace ep
