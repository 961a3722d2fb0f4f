// The experts' products between dispatch and combine: host launchers and the device helpers that
// their kernels share (internal header).
#pragma once

#include "ep_device.h"
#include "ep_internal.h"

namespace ep {

// One grouped FP8 product: rows of E experts (padded [E][C], or packed with `offset`) times each
// expert's weights [n][H]. Outputs: y (bf16, n channels per row), or h_q / h_scale (SwiGLU of the
// n = 2I channels, cast to FP8).
struct ExpertProduct {
    const uint8_t *q;         // row codes, H per row
    const float *scale;       // row scales, H/128 per row
    const int32_t *count;     // [E] rows per expert
    const int32_t *offset;    // packed: first row of each expert; null: padded
    const uint8_t *w_q;       // [E][n][H]
    const float *w_scale;     // [E][ceil(n/128)][H/128]
    uint16_t *y;
    uint8_t *h_q;
    float *h_scale;
    int E, C, rows, H, n;
    int pairs;                // pairs laid out: chooses the grid, nothing else
};

hipError_t launch_expert_gemm_fp8(const ExpertProduct &p, hipStream_t stream);
hipError_t launch_expert_swiglu_fp8(const ExpertProduct &p, hipStream_t stream);

// A whole MoE layer for a few tokens; weights bf16 (scales null) or E4M3 with 128 x 128 scales.
struct MoeLayer {
    const uint16_t *x;        // [T][H] bf16
    const int32_t *idx;       // [T][K]
    const float *topk_w;      // [T][K]
    const void *w13;          // [E][2I][H]: gate rows, then up rows
    const float *w13_scale;   // [E][2I/128][H/128]
    const void *w2;           // [E][H][I]
    const float *w2_scale;    // [E][H/128][I/128]
    uint16_t *h;              // workspace: T*K rows of h, see ep_moe_layer.hip
    float *y;                 // workspace: [T*K][H], above kMoeSmallPairs pairs
    int32_t *named;           // workspace: number of named experts, then {expert, first row, rows, 0} each
    int32_t *order;           // workspace: pair of each row
    uint16_t *out;            // [T][H] bf16
    int T, E, K, H, I;
};

constexpr int kMoePairs = EP_MOE_MAX_PAIRS;

// Up to here the down kernel keeps every pair's y in LDS and needs no list of the named experts and
// no launch for the sum (one token of 8 pairs, H = 4096, I = 1024, FP8: 27 us against 32; 16 pairs 50
// against 55; 32 pairs of H = 2048, I = 768 45.5 against 39, 64 pairs 80 against 62: there the
// many workgroups of the other kernel pay).
constexpr int kMoeSmallPairs = 16;

// Bytes of the layer's workspace: h in two bf16 parts and, above kMoeSmallPairs, y and the lists (4
// words per named expert and one per pair; there are at most as many named experts as pairs).
inline size_t moe_workspace_bytes(size_t pairs, size_t I, size_t H)
{
    return pairs * I * 4 + (pairs > kMoeSmallPairs ? pairs * (H + 5) * 4 + 16 : 0);
}

hipError_t launch_moe_layer(const MoeLayer &p, bool fp8, hipStream_t stream);

#if defined(__HIPCC__)

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Two ways to multiply E4M3 codes. The FP8 matrix instruction aligns each group of products to the
// largest and cuts what lies 14 binary places below it: measured 1.3e-5 (2e-5 with outliers) of the
// result's norm, good enough in front of a rounding to bf16 (2e-3), not in front of an fp32 output.
// The codes as bf16 (every E4M3 value is one) through the bf16 matrix instructions lose nothing above
// fp32's own rounding (1e-8), at half the rate.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes as bf16.
__device__ __forceinline__ bf16x8 bf16_of_e4m3(int c0, int c1)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ i32x8 join(i32x4 lo, i32x4 hi)
{
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// h = g / (1 + exp(-g)) * u. The reciprocal is the hardware's, within one step of fp32, for a
// division's tenth of the instructions. Its result must not be subnormal, for it would be 0: for
// g below -87.3 the sum passes 2^126, and with a large u h is of an ordinary size there. So it is
// taken of a sixteenth of the sum (exact), and its sixteenth by a product, which keeps subnormals.
// The exponential is the hardware's 2^x: rounding its argument gives h a relative error of
// 1.5 |g| + 8 half steps of fp32 at most, which shows where g is far below 0 and h small. Below
// -88.7 exp(-g) is infinite in fp32 and h a zero; g = -inf gives NaN, as -inf / inf does.
__device__ __forceinline__ float swiglu(float g, float u)
{
    const float sum16 = __builtin_fmaf(__expf(-g), 0x1p-4f, 0x1p-4f);
    return g * (__builtin_amdgcn_rcpf(sum16) * 0x1p-4f) * u;
}

// Rows of expert e: first row and number (0 if the counts or offsets leave none in the buffer).
__device__ __forceinline__ void expert_rows(const int32_t *count, const int32_t *offset, int e,
                                            int C, int rows, int &base, int &n)
{
    n = min(max(count[e], 0), C);
    base = offset ? offset[e] : e * C;
    if (offset) {
        if (base < 0 || base >= rows) n = base = 0;
        else n = min(n, rows - base);
    }
}

#endif

}  // namespace ep
