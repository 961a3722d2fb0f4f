// A whole MoE layer for a few tokens on gfx950, in two launches with no receive buffer:
//
//   moe_up_kernel    h[i] = silu(Wg[e] x[t]) * (Wu[e] x[t]) for each pair i = t*K + j, e = idx[i]
//   moe_down_kernel  out[t] = bf16( sum_j w[i] * W2[e] h[i] )
//
// With a few rows per expert the layer reads the chosen experts' weights once and does little
// else, so both kernels stream weight rows from HBM straight into registers as the A operand of
// the bf16 matrix instructions (FP8 codes are converted there, exactly) and keep the pairs' rows
// as the B operand: 16 weight rows x 16 pairs per instruction.
//
// Products are exact and summed in fp32. h goes through the workspace as two bf16 values, hi and
// lo = h - hi (16 significant bits together): one bf16 alone would add as much error as the final
// rounding of out does.
#include "ep_expert.h"

namespace ep {

namespace {

constexpr int kUpWaves = 4;
constexpr int kTileC = 16;                    // output columns per workgroup of the down kernel

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A step along a weight row: 128 bytes, 32 of them per lane (chunks g4 and g4 + 4 of 16 bytes),
// and the same elements of a bf16 row.
template <bool FP8>
struct Step {
    static constexpr int kElems = FP8 ? 128 : 64;
    static constexpr int kMfma = FP8 ? 4 : 2;
};

template <bool FP8>
struct Frag {
    bf16x8 v[Step<FP8>::kMfma];
};

__device__ __forceinline__ bf16x8 as_bf16(i32x4 v) { return __builtin_bit_cast(bf16x8, v); }

template <bool FP8>
__device__ __forceinline__ Frag<FP8> weight_frag(i32x4 a, i32x4 b)
{
    if constexpr (FP8)
        return Frag<FP8>{{bf16_of_e4m3(a[0], a[1]), bf16_of_e4m3(a[2], a[3]),
                          bf16_of_e4m3(b[0], b[1]), bf16_of_e4m3(b[2], b[3])}};
    else
        return Frag<FP8>{{as_bf16(a), as_bf16(b)}};
}

// The lane's elements of one step of a bf16 row starting at byte offset `off` (lane part
// included: g4 * 16 * (FP8 ? 2 : 1) bytes).
template <bool FP8>
__device__ __forceinline__ Frag<FP8> row_frag(const uint8_t *row, uint32_t off)
{
    const i32x4 *p = reinterpret_cast<const i32x4 *>(row + off);
    if constexpr (FP8)
        return Frag<FP8>{{as_bf16(p[0]), as_bf16(p[1]), as_bf16(p[8]), as_bf16(p[9])}};
    else
        return Frag<FP8>{{as_bf16(p[0]), as_bf16(p[4])}};
}

template <bool FP8>
__device__ __forceinline__ f32x4 mfma_frag(const Frag<FP8> &a, const Frag<FP8> &b, f32x4 c)
{
#pragma unroll
    for (int i = 0; i < Step<FP8>::kMfma; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

// h = silu(g) * u.
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// NI: tiles of 16 channels of h per workgroup.
template <bool FP8, int NI>
struct UpShared {
    uint32_t named[EP_MAX_EXPERTS / 32];      // experts that a pair names
    int n;                                    // pairs of this workgroup's expert
    uint16_t pair[kMoePairs];
    f32x4 part[kUpWaves][2 * NI][kWave];      // the wavefronts' sums of one tile of 16 pairs
};

// One pass over the expert's weights for MT tiles of 16 pairs. The wavefronts take the steps along
// H in turn and their sums meet in LDS, in wavefront order.
template <bool FP8, int NI, int MT, int D>
__device__ __forceinline__ void up_pass(UpShared<FP8, NI> &sh, const MoeLayer &p, int e, int c0,
                                        int first, int n)
{
    constexpr int kS = Step<FP8>::kElems;
    const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int row_bytes = FP8 ? p.H : 2 * p.H;
    const uint8_t *w = static_cast<const uint8_t *>(p.w13) + (size_t)e * 2 * p.I * row_bytes;
    uint32_t woff[2][NI], xoff[MT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
            woff[i][ni] = (uint32_t)(i * p.I + c0 + ni * 16 + r16) * row_bytes + g4 * 16;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int t = sh.pair[first + min(mt * 16 + r16, n - 1)] / p.K;
        xoff[mt] = (uint32_t)t * p.H * 2 + g4 * (FP8 ? 32 : 16);
    }
    const uint8_t *x = reinterpret_cast<const uint8_t *>(p.x);
    const int nsteps = p.H / kS;
    const float *ws[2] = {nullptr, nullptr};
    if constexpr (FP8)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            ws[i] = p.w13_scale +
                    ((size_t)e * (2 * p.I >> 7) + ((i * p.I + c0) >> 7)) * (size_t)nsteps;

    f32x4 acc[2][NI][MT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[i][ni][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    i32x4 wf[D][2][NI][2];
    Frag<FP8> xf[D][MT];
    float sw[D][2];
    auto load = [&](int d, int s) {
        const uint8_t *wk = w + (size_t)s * 128, *xk = x + (size_t)s * (kS * 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) {
                wf[d][i][ni][0] = *reinterpret_cast<const i32x4 *>(wk + woff[i][ni]);
                wf[d][i][ni][1] = *reinterpret_cast<const i32x4 *>(wk + woff[i][ni] + 64);
            }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) xf[d][mt] = row_frag<FP8>(xk, xoff[mt]);
        if constexpr (FP8) {
            sw[d][0] = ws[0][s];
            sw[d][1] = ws[1][s];
        }
    };
    if (wave < nsteps) {
#pragma unroll
        for (int d = 0; d < D; ++d) load(d, min(wave + d * kUpWaves, nsteps - 1));
        for (int s = wave; s < nsteps; s += D * kUpWaves) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (s + d * kUpWaves < nsteps) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int ni = 0; ni < NI; ++ni) {
                            const Frag<FP8> a =
                                weight_frag<FP8>(wf[d][i][ni][0], wf[d][i][ni][1]);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                f32x4 &c = acc[i][ni][mt];
                                if constexpr (FP8) {
                                    const f32x4 v = mfma_frag<FP8>(
                                        a, xf[d][mt], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        c[k] = __builtin_fmaf(sw[d][i], v[k], c[k]);
                                } else {
                                    c = mfma_frag<FP8>(a, xf[d][mt], c);
                                }
                            }
                        }
                }
                load(d, min(s + (d + D) * kUpWaves, nsteps - 1));
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) sh.part[wave][i * NI + ni][lane] = acc[i][ni][mt];
        __syncthreads();
        for (int f = threadIdx.x; f < NI * 256; f += kUpWaves * kWave) {
            const int r = f / (NI * 16), c = f % (NI * 16);          // pair, channel
            const int ni = c >> 4, l = ((c >> 2) & 3) * 16 + r, k = c & 3;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int v = 0; v < kUpWaves; ++v) {
                g += reinterpret_cast<const float *>(&sh.part[v][ni][l])[k];
                u += reinterpret_cast<const float *>(&sh.part[v][NI + ni][l])[k];
            }
            if (mt * 16 + r < n) {
                const float h = swiglu(g, u);
                const uint32_t hi = bf16_rne(h);
                const size_t at = (size_t)sh.pair[first + mt * 16 + r] * p.I + c0 + c;
                p.h_hi[at] = (uint16_t)hi;
                // an infinite or NaN h is whole in hi
                const float rest = h - __uint_as_float(hi << 16);
                p.h_lo[at] = (hi & 0x7F80u) == 0x7F80u ? 0 : (uint16_t)bf16_rne(rest);
            }
        }
        __syncthreads();
    }
}

// blockIdx.x: NI * 16 channels of h; blockIdx.y: the number of an expert among those named.
template <bool FP8, int NI>
__global__ __launch_bounds__(kUpWaves *kWave) void moe_up_kernel(MoeLayer p)
{
    __shared__ UpShared<FP8, NI> sh;
    const int lane = threadIdx.x & (kWave - 1);
    const int pairs = p.T * p.K;
    if (threadIdx.x < EP_MAX_EXPERTS / 32) sh.named[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kUpWaves * kWave) {
        const int e = p.idx[i];
        if ((unsigned)e < (unsigned)p.E) atomicOr(&sh.named[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    // the blockIdx.y-th set bit
    const uint32_t word = lane < EP_MAX_EXPERTS / 32 ? sh.named[lane] : 0u;
    const int bits = __popc(word), incl = wave_inclusive_sum(bits);
    const int want = blockIdx.y;
    const uint64_t mine = __ballot(incl - bits <= want && want < incl);
    if (mine == 0) return;                     // fewer experts are named
    const int at = __ffsll((unsigned long long)mine) - 1;
    uint32_t left = (uint32_t)__shfl((int)word, at);
    for (int skip = want - __shfl(incl - bits, at); skip > 0; --skip) left &= left - 1;
    const int e = uniform(at * 32 + __ffs(left) - 1);
    for (int i = threadIdx.x; i < pairs; i += kUpWaves * kWave)
        if (p.idx[i] == e) sh.pair[atomicAdd(&sh.n, 1)] = (uint16_t)i;
    __syncthreads();
    const int n = uniform(sh.n), c0 = blockIdx.x * NI * 16;
    int first = 0;
    while (n - first > 16) {
        up_pass<FP8, NI, 4, 1>(sh, p, e, c0, first, min(n - first, 64));
        first += 64;
    }
    if (first < n) up_pass<FP8, NI, 1, NI == 1 ? 4 : NI == 2 ? 2 : 1>(sh, p, e, c0, first, n - first);
}

// The down kernel's LDS: y of every pair for the workgroup's 16 columns, and the pairs sorted by
// expert.
struct DownShared {
    int32_t count[EP_MAX_EXPERTS], first[EP_MAX_EXPERTS];
    uint16_t named[EP_MAX_EXPERTS];
    uint16_t rank[kMoePairs], pair[kMoePairs];
    int n_named, next;
};

template <bool FP8, int MT, int D>
__device__ __forceinline__ void down_pass(const DownShared &sh, f32x4 *y, const MoeLayer &p, int e,
                                          int c0, int first, int n)
{
    constexpr int kS = Step<FP8>::kElems;
    const int lane = threadIdx.x & (kWave - 1);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int row_bytes = FP8 ? p.I : 2 * p.I;
    const uint8_t *w = static_cast<const uint8_t *>(p.w2) + (size_t)e * p.H * row_bytes;
    const uint32_t woff = (uint32_t)(c0 + r16) * row_bytes + g4 * 16;
    int pair[MT];
    uint32_t hoff[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        pair[mt] = sh.pair[first + min(mt * 16 + r16, n - 1)];
        hoff[mt] = (uint32_t)pair[mt] * p.I * 2 + g4 * (FP8 ? 32 : 16);
    }
    const uint8_t *hi = reinterpret_cast<const uint8_t *>(p.h_hi);
    const uint8_t *lo = reinterpret_cast<const uint8_t *>(p.h_lo);
    const int nsteps = p.I / kS;
    const float *ws = nullptr;
    if constexpr (FP8) ws = p.w2_scale + ((size_t)e * (p.H >> 7) + (c0 >> 7)) * (size_t)nsteps;

    f32x4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    i32x4 wf[D][2];
    Frag<FP8> hf[D][MT][2];
    float sw[D];
    auto load = [&](int d, int s) {
        const uint8_t *wk = w + (size_t)s * 128;
        wf[d][0] = *reinterpret_cast<const i32x4 *>(wk + woff);
        wf[d][1] = *reinterpret_cast<const i32x4 *>(wk + woff + 64);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            hf[d][mt][0] = row_frag<FP8>(hi + (size_t)s * (kS * 2), hoff[mt]);
            hf[d][mt][1] = row_frag<FP8>(lo + (size_t)s * (kS * 2), hoff[mt]);
        }
        if constexpr (FP8) sw[d] = ws[s];
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, min(d, nsteps - 1));
    for (int s = 0; s < nsteps; s += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (s + d < nsteps) {
                const Frag<FP8> a = weight_frag<FP8>(wf[d][0], wf[d][1]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (FP8) {
                        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
                        v = mfma_frag<FP8>(a, hf[d][mt][1], v);
                        v = mfma_frag<FP8>(a, hf[d][mt][0], v);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[mt][k] = __builtin_fmaf(sw[d], v[k], acc[mt][k]);
                    } else {
                        acc[mt] = mfma_frag<FP8>(a, hf[d][mt][1], acc[mt]);
                        acc[mt] = mfma_frag<FP8>(a, hf[d][mt][0], acc[mt]);
                    }
                }
            }
            load(d, min(s + d + D, nsteps - 1));
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        if (mt * 16 + r16 < n) y[pair[mt] * (kTileC / 4) + g4] = acc[mt];
}

// A workgroup: 16 columns of out for all tokens. Its wavefronts take the named experts from a
// counter in LDS; y of every pair meets there, and the weighted sums run over j in order.
template <bool FP8>
__global__ __launch_bounds__(1024) void moe_down_kernel(MoeLayer p)
{
    extern __shared__ f32x4 y[];               // [pairs][16]
    __shared__ DownShared sh;
    const int lane = threadIdx.x & (kWave - 1);
    const int pairs = p.T * p.K, nthreads = blockDim.x;
    for (int e = threadIdx.x; e < p.E; e += nthreads) sh.count[e] = 0;
    if (threadIdx.x == 0) sh.next = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += nthreads) {
        const int e = p.idx[i];
        if ((unsigned)e < (unsigned)p.E) sh.rank[i] = (uint16_t)atomicAdd(&sh.count[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < kWave) {                 // first pair of each expert, and the named experts
        int run = 0, named = 0;
        for (int e0 = 0; e0 < p.E; e0 += kWave) {
            const int e = e0 + lane, c = e < p.E ? sh.count[e] : 0;
            const int incl = wave_inclusive_sum(c);
            const uint64_t some = __ballot(c > 0);
            if (e < p.E) sh.first[e] = run + incl - c;
            if (c > 0) sh.named[named + count_below(some)] = (uint16_t)e;
            run += __shfl(incl, kWave - 1);
            named += __popcll(some);
        }
        if (lane == 0) sh.n_named = named;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += nthreads) {
        const int e = p.idx[i];
        if ((unsigned)e < (unsigned)p.E) sh.pair[sh.first[e] + sh.rank[i]] = (uint16_t)i;
    }
    __syncthreads();

    const int c0 = blockIdx.x * kTileC, n_named = sh.n_named;
    while (true) {
        int a = 0;
        if (lane == 0) a = atomicAdd(&sh.next, 1);
        a = uniform(a);
        if (a >= n_named) break;
        const int e = uniform(sh.named[a]), n = uniform(sh.count[e]);
        int first = uniform(sh.first[e]), left = n;
        while (left > 16) {
            down_pass<FP8, 4, 1>(sh, y, p, e, c0, first, min(left, 64));
            first += 64;
            left -= 64;
        }
        if (left > 0) down_pass<FP8, 1, 2>(sh, y, p, e, c0, first, left);
    }
    __syncthreads();
    const float *yf = reinterpret_cast<const float *>(y);
    for (int f = threadIdx.x; f < p.T * kTileC; f += nthreads) {
        const int t = f / kTileC, c = f % kTileC;
        float acc = 0.0f;
        for (int j = 0; j < p.K; ++j) {
            const int i = t * p.K + j;
            if ((unsigned)p.idx[i] < (unsigned)p.E)
                acc = __builtin_fmaf(p.topk_w[i], yf[i * kTileC + c], acc);
        }
        p.out[(size_t)t * p.H + c0 + c] = (uint16_t)bf16_rne(acc);
    }
}

template <bool FP8>
hipError_t launch_fp8(const MoeLayer &p, hipStream_t stream)
{
    const int pairs = p.T * p.K;
    const int named = pairs < p.E ? pairs : p.E;       // at most
    const dim3 block(kUpWaves * kWave);
    const long tiles = (long)named * (p.I / 16);
    hipError_t e;
    if (tiles >= 4096)
        e = launch(moe_up_kernel<FP8, 4>, dim3(p.I / 64, named), block, 0, stream, p);
    else if (tiles >= 1024)
        e = launch(moe_up_kernel<FP8, 2>, dim3(p.I / 32, named), block, 0, stream, p);
    else
        e = launch(moe_up_kernel<FP8, 1>, dim3(p.I / 16, named), block, 0, stream, p);
    if (e != hipSuccess) return e;
    const int waves = named < 4 ? 4 : named > 16 ? 16 : named;
    return launch(moe_down_kernel<FP8>, dim3(p.H / kTileC), dim3(waves * kWave),
                  (size_t)pairs * kTileC * sizeof(float), stream, p);
}

}  // namespace

hipError_t launch_moe_layer(const MoeLayer &p, bool fp8, hipStream_t stream)
{
    return fp8 ? launch_fp8<true>(p, stream) : launch_fp8<false>(p, stream);
}

}  // namespace ep
