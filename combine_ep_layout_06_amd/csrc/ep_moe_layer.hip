// A whole MoE layer for a few tokens on gfx950, in two or three launches with no receive buffer:
//
//   moe_up_kernel    h[i] = silu(Wg[e] x[t]) * (Wu[e] x[t]) for each pair i = t*K + j, e = idx[i]
//   moe_small_down_kernel  out[t] = bf16( sum_j w[i] * W2[e] h[i] )
// or, above kMoeSmallPairs pairs,
//   moe_down_kernel  y[i] = W2[e] h[i]
//   moe_sum_kernel   out[t] = bf16( sum_j w[i] * y[i] )
//
// With a few rows per expert the layer reads the chosen experts' weights once and does little
// else, so both kernels stream weight rows from HBM straight into registers as the A operand of
// the bf16 matrix instructions (FP8 codes are converted there, exactly) and keep the pairs' rows
// as the B operand: 16 weight rows x 16 pairs per instruction.
//
// Products are exact and summed in fp32. h goes through the workspace as two bf16 values, hi and
// lo = h - hi (16 significant bits together): one bf16 alone would add as much error as the final
// rounding of out does. It is laid out for the down kernel's loads: an expert's n rows together,
// [I/8 chunks][hi, lo][n rows][8 channels], so that neighbouring lanes (rows, in the matrix
// instruction's order) read neighbouring 16 bytes; row-major, every lane's 16 bytes took a cache
// access of its own, and that bounded the down kernel (128 tokens, FP8: 172 us).
#include "ep_expert.h"

namespace ep {

namespace {

constexpr int kUpWaves = 4;
static_assert(kMoeSmallPairs <= 16, "a wavefront per pair, one tile of rows per expert");

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

// The pairs of one expert: its rows are `first` .. first + n - 1 of h (experts in order of their
// ids, pairs in order), `mine` lane l's pair: that of row l.
struct Rows {
    int first, n;
};

// At most kMoeSmallPairs pairs: lane l holds the id of pair l (-1: none). False if pair i names no expert or one
// that an earlier pair names; else the expert's rows, and in `pair` the lane's pair: lane r gets the
// pair of row r (r < n).
__device__ __forceinline__ bool small_rows(int id, int E, int i, int &e, Rows &r, int &pair)
{
    e = __builtin_amdgcn_readlane(id, i);
    if ((unsigned)e >= (unsigned)E) return false;
    const uint64_t same = __ballot(id == e);
    if (same & ((1ull << i) - 1)) return false;
    r.n = __popcll(same);
    r.first = __popcll(__ballot(id >= 0 && id < e));
    const int lane = threadIdx.x & (kWave - 1);
    const int to = id == e ? count_below(same) : r.n + count_below(~same);
    pair = __builtin_amdgcn_ds_permute(to * 4, lane);
    return true;
}

// NI: tiles of 16 channels of h per workgroup.
template <int NI>
struct UpShared {
    uint32_t named[EP_MAX_EXPERTS / 32];      // experts that a pair names
    int first, n;                             // rows of this workgroup's expert
    uint16_t pair[kMoePairs];                 // their pairs
    f32x4 part[kUpWaves][2 * NI][kWave];      // the wavefronts' sums of one tile of 16 pairs
};

// One pass over the expert's weights for MT tiles of 16 pairs, rows row0 .. row0 + n - 1 of its
// rows.n. The wavefronts take the steps along H in turn and their sums meet in LDS, in wavefront
// order.
template <bool FP8, int NI, int MT, int D>
__device__ __forceinline__ void up_pass(UpShared<NI> &sh, const MoeLayer &p, int e, int c0,
                                        const Rows &rows, int row0, int n)
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
        const int t = sh.pair[row0 + min(mt * 16 + r16, n - 1)] / p.K;
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
                if (s + (d + D) * kUpWaves < nsteps) load(d, s + (d + D) * kUpWaves);
            }
        }
    }
    uint16_t *h_e = p.h + (size_t)rows.first * 2 * p.I;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) sh.part[wave][i * NI + ni][lane] = acc[i][ni][mt];
        __syncthreads();
        for (int f = threadIdx.x; f < NI * 256; f += kUpWaves * kWave) {
            // 8 channels of a row next to each other, then the rows
            const int c = (f & 7) | (f >> 7) << 3, r = (f >> 3) & 15;
            const int ni = c >> 4, l = ((c >> 2) & 3) * 16 + r, k = c & 3;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int v = 0; v < kUpWaves; ++v) {
                g += reinterpret_cast<const float *>(&sh.part[v][ni][l])[k];
                u += reinterpret_cast<const float *>(&sh.part[v][NI + ni][l])[k];
            }
            if (mt * 16 + r < n) {
                const float h = swiglu(g, u);
                uint32_t hi = bf16_rne(h);
                // a finite h that rounds to infinity keeps the largest finite value in hi and the
                // rest in lo; an infinite or NaN h is whole in hi
                if ((hi & 0x7FFFu) == 0x7F80u && __builtin_isfinite(h)) --hi;
                const float rest = h - __uint_as_float(hi << 16);
                const int ch = c0 + c;
                uint16_t *at = h_e + ((size_t)(ch >> 3) * 2 * rows.n + row0 + mt * 16 + r) * 8 + (ch & 7);
                at[0] = (uint16_t)hi;
                at[(size_t)rows.n * 8] = (hi & 0x7F80u) == 0x7F80u ? 0 : (uint16_t)bf16_rne(rest);
            }
        }
        __syncthreads();
    }
}

// blockIdx.x: NI * 16 channels of h; blockIdx.y: the number of an expert among those named (SMALL,
// at most kMoeSmallPairs pairs: a pair, whose expert is taken if no earlier pair names it).
template <bool FP8, int NI, bool SMALL>
__global__ __launch_bounds__(kUpWaves *kWave, 2) void moe_up_kernel(MoeLayer p)
{
    __shared__ UpShared<NI> sh;
    const int lane = threadIdx.x & (kWave - 1);
    const int pairs = p.T * p.K, c0 = blockIdx.x * NI * 16;
    Rows rows;
    int e;
    if constexpr (SMALL) {
        const int id = lane < pairs ? p.idx[lane] : -1;
        int pair;
        if (!small_rows(id, p.E, blockIdx.y, e, rows, pair)) return;
        if (threadIdx.x < kWave) sh.pair[lane] = (uint16_t)pair;
        __syncthreads();
    } else {
        if (threadIdx.x < EP_MAX_EXPERTS / 32) sh.named[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < pairs; i += kUpWaves * kWave) {
            const int v = p.idx[i];
            if ((unsigned)v < (unsigned)p.E) atomicOr(&sh.named[v >> 5], 1u << (v & 31));
        }
        __syncthreads();
        // the blockIdx.y-th set bit
        const uint32_t word = lane < EP_MAX_EXPERTS / 32 ? sh.named[lane] : 0u;
        const int bits = __popc(word), incl = wave_inclusive_sum(bits);
        const int want = blockIdx.y;
        const uint64_t mine = __ballot(incl - bits <= want && want < incl);
        if (blockIdx.x == 0 && want == 0 && threadIdx.x == kWave - 1) p.named[0] = incl;
        if (mine == 0) return;                 // fewer experts are named
        const int at = __ffsll((unsigned long long)mine) - 1;
        uint32_t left = (uint32_t)__shfl((int)word, at);
        for (int skip = want - __shfl(incl - bits, at); skip > 0; --skip) left &= left - 1;
        e = uniform(at * 32 + __ffs(left) - 1);
        if (threadIdx.x < kWave) {             // the expert's pairs in order, and the rows before
            int n = 0, first = 0;
            for (int i0 = 0; i0 < pairs; i0 += kWave) {
                const int i = i0 + lane, v = i < pairs ? p.idx[i] : -1;
                const uint64_t same = __ballot(v == e);
                if (v == e) sh.pair[n + count_below(same)] = (uint16_t)i;
                n += __popcll(same);
                first += __popcll(__ballot(v >= 0 && v < e));
            }
            if (lane == 0) {
                sh.n = n;
                sh.first = first;
            }
        }
        __syncthreads();
        rows = Rows{uniform(sh.first), uniform(sh.n)};
        if (blockIdx.x == 0) {                 // the lists for the down kernel
            if (threadIdx.x == 0)
                reinterpret_cast<int4 *>(p.named)[1 + want] = int4{e, rows.first, rows.n, 0};
            for (int r = threadIdx.x; r < rows.n; r += kUpWaves * kWave)
                p.order[rows.first + r] = sh.pair[r];
        }
    }
    // steps in flight: with one tile all that a wavefront has of H = 2048; with two, 2 (FP8) and 3
    // (bf16) are best (1: 32 tokens bf16 222 us, 3: 207 us; 128 tokens FP8 171 us with 2, 180 with 3)
    constexpr int kAhead = NI == 1 ? (FP8 ? 4 : 8) : FP8 ? 2 : 3;
    int row0 = 0;
    if constexpr (!SMALL)
        while (rows.n - row0 > 16) {
            up_pass<FP8, NI, 2, 1>(sh, p, e, c0, rows, row0, min(rows.n - row0, 32));
            row0 += 32;
        }
    if (row0 < rows.n)
        up_pass<FP8, NI, 1, kAhead>(sh, p, e, c0, rows, row0, rows.n - row0);
}

// 16 output columns (weight rows) of an expert for MT tiles of 16 of its rows; the sums go to row
// `pair` of y. The loads of the weights run DW steps ahead, those of h DH (DW a multiple of it).
template <bool FP8, int MT, int DW, int DH>
__device__ __forceinline__ void down_pass(float *y, int stride, const MoeLayer &p, int e, int c0,
                                          const Rows &rows, int row0, const int (&pair)[MT])
{
    constexpr int kS = Step<FP8>::kElems;
    const int lane = threadIdx.x & (kWave - 1);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int row_bytes = FP8 ? p.I : 2 * p.I;
    const uint8_t *w = static_cast<const uint8_t *>(p.w2) + (size_t)e * p.H * row_bytes;
    const uint32_t woff = (uint32_t)(c0 + r16) * row_bytes + g4 * 16;
    const uint8_t *h = reinterpret_cast<const uint8_t *>(p.h + (size_t)rows.first * 2 * p.I);
    const int n = rows.n, nsteps = p.I / kS;
    // a lane's place in its chunks of h: chunk c of a step is 2 * n * 16 bytes further per c
    uint32_t hoff[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        hoff[mt] = (uint32_t)((FP8 ? 2 * g4 : g4) * 2 * n + row0 + min(mt * 16 + r16, n - 1 - row0)) * 16;
    const float *ws = nullptr;
    if constexpr (FP8) ws = p.w2_scale + ((size_t)e * (p.H >> 7) + (c0 >> 7)) * (size_t)nsteps;

    f32x4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    i32x4 wf[DW][2];
    float sw[DW];
    auto load = [&](int d, int s) {
        const uint8_t *wk = w + (size_t)s * 128;
        wf[d][0] = *reinterpret_cast<const i32x4 *>(wk + woff);
        wf[d][1] = *reinterpret_cast<const i32x4 *>(wk + woff + 64);
        if constexpr (FP8) sw[d] = ws[s];
    };
    Frag<FP8> hf[DH][MT][2];                   // lo, hi
    auto load_h = [&](int d, int s) {
#pragma unroll
        for (int i = 0; i < Step<FP8>::kMfma; ++i) {
            // the 8 channels that the lane's i-th 8 codes (FP8) or i-th 16 bytes meet
            const int c = s * (kS / 8) + (FP8 ? (i >> 1) * 8 + (i & 1) : i * 4);
            const uint8_t *hi = h + (size_t)c * 2 * n * 16, *lo = hi + n * 16;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                hf[d][mt][1].v[i] = as_bf16(*reinterpret_cast<const i32x4 *>(hi + hoff[mt]));
                hf[d][mt][0].v[i] = as_bf16(*reinterpret_cast<const i32x4 *>(lo + hoff[mt]));
            }
        }
    };
#pragma unroll
    for (int d = 0; d < DW; ++d) load(d, min(d, nsteps - 1));
#pragma unroll
    for (int d = 0; d < DH; ++d) load_h(d, min(d, nsteps - 1));
    for (int s = 0; s < nsteps; s += DW) {
#pragma unroll
        for (int d = 0; d < DW; ++d) {
            if (s + d < nsteps) {
                const Frag<FP8> a = weight_frag<FP8>(wf[d][0], wf[d][1]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (FP8) {
                        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
                        v = mfma_frag<FP8>(a, hf[d % DH][mt][0], v);
                        v = mfma_frag<FP8>(a, hf[d % DH][mt][1], v);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[mt][k] = __builtin_fmaf(sw[d], v[k], acc[mt][k]);
                    } else {
                        acc[mt] = mfma_frag<FP8>(a, hf[d % DH][mt][0], acc[mt]);
                        acc[mt] = mfma_frag<FP8>(a, hf[d % DH][mt][1], acc[mt]);
                    }
                }
            }
            if (s + d + DH < nsteps) load_h(d % DH, s + d + DH);
            if (s + d + DW < nsteps) load(d, s + d + DW);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        if (row0 + mt * 16 + r16 < n)
            *reinterpret_cast<f32x4 *>(y + (size_t)pair[mt] * stride + g4 * 4) = acc[mt];
}

// At most kMoeSmallPairs pairs. A workgroup: 16 columns of out for all tokens (8, for twice the
// workgroups, won nowhere: one token, H = 4096, FP8 22.3 against 19.4 us; H = 1024 13.9 against 13.6).
// A wavefront takes a pair's expert if no earlier pair names it; y of every pair meets in LDS, and
// the weighted sums run over j in order.
constexpr int kCols = 16;

template <bool FP8>
__global__ __launch_bounds__(kMoeSmallPairs *kWave) void moe_small_down_kernel(MoeLayer p)
{
    __shared__ float y[kMoeSmallPairs * kCols], weight[kMoeSmallPairs];
    __shared__ bool names[kMoeSmallPairs];
    const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
    const int pairs = p.T * p.K, nthreads = blockDim.x, c0 = blockIdx.x * kCols;
    const int id = lane < pairs ? p.idx[lane] : -1;
    if (threadIdx.x < kMoeSmallPairs) {
        names[lane] = (unsigned)id < (unsigned)p.E;
        weight[lane] = lane < pairs ? p.topk_w[lane] : 0.0f;
    }
    Rows rows;
    int e, pair;
    if (wave < pairs && small_rows(id, p.E, wave, e, rows, pair)) {
        const int of[1] = {__shfl(pair, lane & 15)};
        down_pass<FP8, 1, 4, 1>(y, kCols, p, e, c0, rows, 0, of);
    }
    __syncthreads();
    for (int f = threadIdx.x; f < p.T * kCols; f += nthreads) {
        const int t = f / kCols, c = f % kCols;
        float acc = 0.0f;
        for (int j = 0; j < p.K; ++j) {
            const int i = t * p.K + j;
            if (names[i]) acc = __builtin_fmaf(weight[i], y[i * kCols + c], acc);
        }
        p.out[(size_t)t * p.H + c0 + c] = (uint16_t)bf16_rne(acc);
    }
}

// blockIdx.x: 64 columns, 16 per wavefront; blockIdx.y: the number of a named expert. y [pair][H].
// Four workgroups per CU with 3 steps of weights in flight each, since a workgroup is short and waits
// for its lists and its first loads (128 tokens FP8: 159 us for the layer; two workgroups with 6
// steps 171 us).
template <bool FP8>
__global__ __launch_bounds__(4 * kWave, 4) void moe_down_kernel(MoeLayer p)
{
    const int a = blockIdx.y, r16 = threadIdx.x & 15;
    if (a >= p.named[0]) return;
    const int4 v = reinterpret_cast<const int4 *>(p.named)[1 + a];
    const int e = uniform(v.x), c0 = blockIdx.x * 64 + uniform(threadIdx.x / kWave) * 16;
    const Rows rows{uniform(v.y), uniform(v.z)};
    int row0 = 0;
    while (rows.n - row0 > 16) {
        int of[2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
            of[mt] = p.order[rows.first + min(row0 + mt * 16 + r16, rows.n - 1)];
        down_pass<FP8, 2, 1, 1>(p.y + c0, p.H, p, e, c0, rows, row0, of);
        row0 += 32;
    }
    if (row0 < rows.n) {
        const int of[1] = {p.order[rows.first + min(row0 + r16, rows.n - 1)]};
        down_pass<FP8, 1, 3, 1>(p.y + c0, p.H, p, e, c0, rows, row0, of);
    }
}

__global__ __launch_bounds__(256) void moe_sum_kernel(MoeLayer p)
{
    const int per = p.H / 4, f = blockIdx.x * 256 + threadIdx.x;
    if (f >= p.T * per) return;
    const int t = f / per, c = (f - t * per) * 4;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < p.K; j0 += 8) {      // 8 pairs in flight; past the last one, it again
        f32x4 v[8];
        float w[8];
        bool names[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = t * p.K + min(j0 + j, p.K - 1);
            names[j] = j0 + j < p.K && (unsigned)p.idx[i] < (unsigned)p.E;
            w[j] = p.topk_w[i];
            v[j] = *reinterpret_cast<const f32x4 *>(p.y + (size_t)i * p.H + c);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                acc[k] = names[j] ? __builtin_fmaf(w[j], v[j][k], acc[k]) : acc[k];
    }
    uint2 o;
    o.x = bf16_rne(acc[0]) | (bf16_rne(acc[1]) << 16);
    o.y = bf16_rne(acc[2]) | (bf16_rne(acc[3]) << 16);
    *reinterpret_cast<uint2 *>(p.out + (size_t)t * p.H + c) = o;
}

template <bool FP8, bool SMALL>
hipError_t launch_layer(const MoeLayer &p, hipStream_t stream)
{
    const int pairs = p.T * p.K;
    const int named = SMALL ? pairs : pairs < p.E ? pairs : p.E;       // at most
    const dim3 block(kUpWaves * kWave);
    // 32 channels of h per workgroup, 16 where that would leave the chip half empty (2 tokens of 8
    // experts, I = 768, FP8: 27.2 us with 16, 28.6 with 32; 16 tokens: 109 and 90; 64 held more
    // registers and lost: 32 tokens bf16 227 against 212 us)
    const long tiles = (long)named * (p.I / 16);
    hipError_t e;
    if (tiles >= 1024)
        e = launch(moe_up_kernel<FP8, 2, SMALL>, dim3(p.I / 32, named), block, 0, stream, p);
    else
        e = launch(moe_up_kernel<FP8, 1, SMALL>, dim3(p.I / 16, named), block, 0, stream, p);
    if (e != hipSuccess) return e;
    if constexpr (SMALL) {
        const int waves = pairs < 4 ? 4 : pairs;
        return launch(moe_small_down_kernel<FP8>, dim3(p.H / kCols), dim3(waves * kWave), 0, stream, p);
    } else {
        e = launch(moe_down_kernel<FP8>, dim3(p.H / 64, named), dim3(4 * kWave), 0, stream, p);
        if (e != hipSuccess) return e;
        const int64_t quads = (int64_t)p.T * (p.H / 4);
        return launch(moe_sum_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, p);
    }
}

}  // namespace

hipError_t launch_moe_layer(const MoeLayer &p, bool fp8, hipStream_t stream)
{
    if (p.T * p.K <= kMoeSmallPairs)
        return fp8 ? launch_layer<true, true>(p, stream) : launch_layer<false, true>(p, stream);
    return fp8 ? launch_layer<true, false>(p, stream) : launch_layer<false, false>(p, stream);
}

}  // namespace ep
