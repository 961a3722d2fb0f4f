// The forward products for few rows on gfx950 (a decode step, one token): bound by reading the weights
// once, and by how soon enough of the read is under way.
//
// A workgroup takes 16 columns of the output (SwiGLU: the same 16 gate and 16 up columns) for up to
// 16 * MT rows of one expert, its 8 wavefronts an eighth of the sum each: so also a narrow product has
// a workgroup for every CU, and all of them read at once. Weights and rows go from memory to registers
// in the order of the 16 x 16 x 32 matrix instruction (16 rows, 64 bytes of each), kAhead steps ahead;
// the wavefronts' sums meet in LDS, in ascending order.
#include "ep_product.h"

#include <algorithm>
#include <cmath>

namespace ep {

namespace {

constexpr int kThreads = 512;
constexpr int kCols = 16;          // columns of a workgroup
constexpr int kMostGroups = 32768; // workgroups of a column; they take more groups in turn

namespace to { constexpr int kBf16 = 0, kSwiglu = 1, kLinear = 2; }

#if defined(__HIP_DEVICE_COMPILE__)

constexpr int kWaves = kThreads / kWave;
constexpr int kStep = 32;          // sum indexes of a matrix instruction
constexpr int kAhead = 8;          // of them loaded together

// The group of rows number `group` of all experts' groups of at most `size` rows: expert, first row, rows,
// and how many groups there are.
struct Group {
    int e, row0, n, of;
};

__device__ __forceinline__ Group find_group(int group, int size)
{
    const auto &p = argument();
    __shared__ int32_t wave_sum[kWaves];
    __shared__ Group found;
    constexpr int kPer = EP_MAX_EXPERTS / kThreads;
    const int lane = lane_now(), wave = uniform(threadIdx.x / kWave);
    const int e0 = (wave * kWave + lane) * kPer;
    int base[kPer], n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        base[i] = n[i] = 0;
        if (e0 + i < p.E) expert_rows(p.count, p.offset, e0 + i, p.C, p.rows, base[i], n[i]);
        sum += (n[i] + size - 1) / size;
    }
    const int incl = wave_inclusive_sum(sum);
    if (lane == kWave - 1) wave_sum[wave] = incl;
    __syncthreads();
    int at = group - (incl - sum), of = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at -= wave_sum[w];
        of += wave_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int groups = (n[i] + size - 1) / size;
        if (at >= 0 && at < groups) found = Group{e0 + i, base[i] + at * size, min(n[i] - at * size, size), of};
        at -= groups;
    }
    __syncthreads();
    // the number also where there is no such group
    return Group{uniform(found.e), uniform(found.row0), uniform(found.n), uniform(of)};
}

template <int O, int MT>
struct FewShared {
    f32x4 meet[kWaves][O == to::kSwiglu ? 2 : 1][MT][kWave];
};

template <int O, int MT>
__device__ __forceinline__ void few_rows(const Group &g, FewShared<O, MT> &sh)
{
    constexpr int kMats = O == to::kSwiglu ? 2 : 1;
    const auto &p = argument();                // nothing is kept from one group to the next
    const int lane = lane_now(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int width = O == to::kSwiglu ? p.n / 2 : p.n;
    const int c0 = blockIdx.x * kCols;
    const int i16 = lane & 15, chunk = (lane >> 4) * 8;
    // a wavefront's steps of the sum
    const int steps = (p.k + kStep - 1) / kStep, per = (steps + kWaves - 1) / kWaves;
    const int s0 = wave * per, s1 = min(s0 + per, steps);
    const uint16_t *w[kMats], *x[MT];
#pragma unroll
    for (int m = 0; m < kMats; ++m)
        w[m] = p.w + ((size_t)g.e * p.n + m * width + min(c0 + i16, width - 1)) * p.k + chunk;
#pragma unroll
    for (int t = 0; t < MT; ++t) x[t] = p.x + (size_t)(g.row0 + min(t * 16 + i16, g.n - 1)) * p.k + chunk;

    f32x4 acc[kMats][MT] = {};
    for (int s = s0; s < s1; s += kAhead) {
        // a wavefront's end of the sum and the row's end: zeros from there on
        const int end = min(s1 * kStep, p.k) - chunk, k0 = s * kStep;
        bf16x8 wf[kAhead][kMats], xf[kAhead][MT];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + i * kStep;
#pragma unroll
            for (int m = 0; m < kMats; ++m)
                wf[i][m] = k < end ? __builtin_nontemporal_load(reinterpret_cast<const bf16x8 *>(w[m] + k))
                                   : bf16x8{};
#pragma unroll
            for (int t = 0; t < MT; ++t)
                xf[i][t] = k < end ? *reinterpret_cast<const bf16x8 *>(x[t] + k) : bf16x8{};
        }
        if constexpr (MT < 4) __builtin_amdgcn_sched_barrier(0);     // every load before the first product
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i][m], xf[i][t], acc[m][t], 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int t = 0; t < MT; ++t) sh.meet[wave][m][t][lane] = acc[m][t];
    __syncthreads();
    // a lane's four sums are columns (lane >> 4) * 4 .. of row lane & 15
    const int t = wave, r = t * 16 + i16, c = c0 + (lane >> 4) * 4;
    if (t >= MT || r >= g.n || c >= width) return;
    f32x4 v[kMats];
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
        v[m] = sh.meet[0][m][t][lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v[m] += sh.meet[i][m][t][lane];
    }
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    auto four = [](f32x4 f) {
        return u32x2{__builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[0], (__bf16)f[1]}),
                     __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[2], (__bf16)f[3]})};
    };
    auto put = [](uint16_t *to, u32x2 d) { *reinterpret_cast<u32x2 *>(to) = d; };
    auto add = [](f32x4 &f, const uint16_t *from) {
        const u32x2 d = *reinterpret_cast<const u32x2 *>(from);
        f += f32x4{bf16_lo(d[0]), bf16_hi(d[0]), bf16_lo(d[1]), bf16_hi(d[1])};
    };
    const size_t row = (size_t)g.row0 + r;
    uint16_t *out = (uint16_t *)p.out + row * width + c;
    if constexpr (O == to::kSwiglu) {
        if (p.out2) {
            put(p.out2 + row * p.n + c, four(v[0]));
            put(p.out2 + row * p.n + width + c, four(v[1]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[0][i] = swiglu(v[0][i], v[1][i]);
    } else if constexpr (O == to::kLinear) {
        if (p.bias) add(v[0], p.bias + c);
        if (p.out2) put(p.out2 + row * p.n + c, four(v[0]));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[0][i] = activate(p.act, v[0][i]);
        if (p.in) add(v[0], p.in + row * p.n + c);
    }
    put(out, four(v[0]));
}

#endif

template <int O, int MT>
__global__ __launch_bounds__(kThreads) void few_rows_kernel(Product p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ FewShared<O, MT> sh;
    constexpr int kSize = kCols * MT;
    for (int group = blockIdx.y;; group += gridDim.y) {
        Group g;
        if (p.count) g = find_group(group, kSize);
        else g = Group{0, group * kSize, min(p.C - group * kSize, kSize), (p.C + kSize - 1) / kSize};
        if (group >= g.of) break;
        few_rows<O, MT>(g, sh);
        if (group + (int)gridDim.y >= g.of) break;
        __syncthreads();                       // the meeting place is free again
    }
#else
    (void)p;
#endif
}

template <int O, int MT>
hipError_t launch_few(const Product &p, hipStream_t stream)
{
    const int width = O == to::kSwiglu ? p.n / 2 : p.n, size = kCols * MT;
    const int groups = p.count ? p.pairs / size + (p.pairs < p.E ? p.pairs : p.E) : (p.C + size - 1) / size;
    return launch(few_rows_kernel<O, MT>, dim3((width + kCols - 1) / kCols, std::min(groups, kMostGroups)),
                  dim3(kThreads), 0, stream, p);
}

// 16 rows that a workgroup takes together, so many times: for the mean of the experts that the rows can
// be spread over.
int row_tiles(const Product &p)
{
    const int mean = p.pairs / (p.pairs < p.E ? p.pairs : p.E);
    return mean <= 16 ? 1 : mean <= 32 ? 2 : 4;
}

template <int O>
hipError_t launch_by_rows(const Product &p, hipStream_t stream)
{
    switch (row_tiles(p)) {
    case 1: return launch_few<O, 1>(p, stream);
    case 2: return launch_few<O, 2>(p, stream);
    default: return launch_few<O, 4>(p, stream);
    }
}

}  // namespace

// Both kernels' times in microseconds, from what they read, for rows spread evenly over the experts.
// Tiles: a block of 64 of the sum takes 0.65 for 64 rows, a round of 256 workgroups at a time, and the
// weights come at 4.9 TB/s. Few rows: every workgroup reads its weights and its rows, at 7.3 TB/s
// together, and costs 0.0025. Measured (tiles, few rows): one matrix of 4096 x 4096, 1 row 42, 9, 64
// rows 43, 24, 96 rows 43, 40, 128 rows 43, 46; 1024 x 2048, 256 rows 25, 12; 16384 x 4096, 16 rows 62,
// 39, 64 rows 64, 94; 128 experts of 1536 x 2048, 8 rows 25, 12, 64 rows 80, 68, 256 rows 157, 149,
// 1024 rows 180, 213; of 2048 x 768, 8 rows 13, 9, 32 rows 20, 27; 16 of 4096 x 4096, 32 rows 109, 73.
bool few_rows(const Product &p, bool swiglu)
{
    const double experts = p.count ? p.E * (1.0 - std::pow(1.0 - 1.0 / p.E, p.pairs)) : 1.0;
    const double mean = p.pairs / experts, k = p.k;
    const int size = kCols * row_tiles(p);
    const double weights = experts * p.n * k * 2.0;
    const double rounds = std::ceil(experts * std::ceil(mean / 64) * std::ceil(p.n / 256.0) / 256);
    const double tiles = std::max(8.0 + rounds * std::ceil(k / 64) * 0.65, 4.0 + weights / 4.9e6);
    const double groups = std::ceil(mean / size), columns = std::ceil(p.n / 16.0) / (swiglu ? 2 : 1);
    const double few = 8.0 + (groups * weights + columns * p.pairs * k * 2.0) / 7.3e6 +
                       experts * groups * columns * 0.0025;
    return few < tiles;
}

hipError_t launch_few_gemm(const Product &p, hipStream_t stream)
{
    return launch_by_rows<to::kBf16>(p, stream);
}

hipError_t launch_few_swiglu(const Product &p, hipStream_t stream)
{
    return launch_by_rows<to::kSwiglu>(p, stream);
}

hipError_t launch_few_linear(const Product &p, hipStream_t stream)
{
    return launch_by_rows<to::kLinear>(p, stream);
}

}  // namespace ep
