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

hipError_t launch_combine_grad(const ep_shape_t &s, const uint16_t *dout, const uint16_t *y,
                               const int32_t *idx, const int32_t *slot, const float *w, uint16_t *dy,
                               float *dw, hipStream_t stream, RowMap map = RowMap());

// Rows whose columns' sums a workgroup of the activation's gradient takes; grid.y holds 65535 of them.
constexpr int kLinearGradRows = 64;

// dz = bf16(dout * act'(z)) (not written without an activation) and dbias, the columns' sums of the
// unrounded dz, through `part`: ceil(T / kLinearGradRows) rows of N.
hipError_t launch_act_grad(const uint16_t *dout, const uint16_t *z, uint16_t *dz, float *part,
                           float *dbias, int T, int N, int act, hipStream_t stream);

}  // namespace ep
