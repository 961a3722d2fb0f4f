// The products for few rows on gfx950 (a decode step, one token), forward and dgrad, bound by reading the
// weights once, and by how soon enough of the read is under way; and products of few tiles.
//
// A workgroup takes 16 columns of the output (SwiGLU: the same 16 gate and 16 up columns) for up to
// 16 * MT rows of one expert, its 8 wavefronts an eighth of the sum each: so also a narrow product has
// a workgroup for every CU, and all of them read at once. Weights and rows go from memory to registers
// in the order of the 16 x 16 x 32 matrix instruction (16 rows, 64 bytes of each), kAhead steps ahead;
// the wavefronts' sums meet in LDS, in ascending order.
//
// Of dgrad's weights [k][n] a column's sum indexes lie rows apart. Its workgroups take 64 columns, and
// each wavefront loads 32 rows of them (128 bytes a row) at a time straight into a ring of LDS of its
// own, from which the transposing read gives the matrix instruction its operand: 64 rows x 4096 x 4096
// 48 -> 20 us, one row 47 -> 11 (the weights at 4.74 TB/s: 7).
//
// Products of more rows with few tiles are made in squares of 64 x 64 in the same way: 1024 rows x 1024 x
// 4096 43 -> 24 us. And weights' gradients of few tiles with long sums, an expert's rows dealt out to the eight
// wavefronts of one workgroup: 8192 rows, 1024 x 1024 93 -> 35 us, 64 x 64 (one workgroup, one CU busy) 89 -> 22,
// in proportion to the rows from there on.
#include "ep_product.h"

#include <algorithm>
#include <cmath>

namespace ep {

namespace {

constexpr int kThreads = 512;
constexpr int kCols = 16;          // columns of a workgroup
constexpr int kMostGroups = 32768; // workgroups of a column; they take more groups in turn

namespace to { constexpr int kBf16 = 0, kSwiglu = 1, kLinear = 2, kSwigluGrad = 3, kF32 = 4; }

__host__ __device__ __forceinline__ int groups_of(int rows, int size)
{
    return ((uint32_t)rows + size - 1) / size;
}

#if defined(__HIP_DEVICE_COMPILE__)

constexpr int kWaves = kThreads / kWave;
constexpr int kStep = 32;          // sum indexes of a matrix instruction
constexpr int kAhead = 8;          // of them loaded together
constexpr int kSquareSlot = 8192;  // a step of both operands of a square
constexpr int kSquareRing = 2;     // such slots of a wavefront

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
        sum += groups_of(n[i], size);
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
        const int groups = groups_of(n[i], size);
        if (at >= 0 && at < groups) found = Group{e0 + i, base[i] + at * size, min(n[i] - at * size, size), of};
        at -= groups;
    }
    __syncthreads();
    // the number also where there is no such group
    return Group{uniform(found.e), uniform(found.row0), uniform(found.n), uniform(of)};
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void put_four(uint16_t *to, f32x4 v)
{
    *reinterpret_cast<u32x2 *>(to) = u32x2{__builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[0], (__bf16)v[1]}),
                                           __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2], (__bf16)v[3]})};
}

__device__ __forceinline__ void add_four(f32x4 &v, const uint16_t *from)
{
    const u32x2 d = *reinterpret_cast<const u32x2 *>(from);
    v += f32x4{bf16_lo(d[0]), bf16_hi(d[0]), bf16_lo(d[1]), bf16_hi(d[1])};
}

// The output's columns c .. c + 3 of a row, from their sums.
template <int O>
__device__ __forceinline__ void put_linear(const Product &p, size_t row, int c, f32x4 v)
{
    if constexpr (O == to::kLinear) {
        if (p.bias) add_four(v, p.bias + c);
        if (p.out2) put_four(p.out2 + row * p.n + c, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(p.act, v[i]);
        if (p.in) add_four(v, p.in + row * p.n + c);
    }
    put_four((uint16_t *)p.out + row * p.n + c, v);
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
    const size_t row = (size_t)g.row0 + r;
    if constexpr (O == to::kSwiglu) {
        if (p.out2) {
            put_four(p.out2 + row * p.n + c, v[0]);
            put_four(p.out2 + row * p.n + width + c, v[1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[0][i] = swiglu(v[0][i], v[1][i]);
        put_four((uint16_t *)p.out + row * width + c, v[0]);
    } else {
        put_linear<O>(p, row, c, v[0]);
    }
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
        else g = Group{0, group * kSize, min(p.C - group * kSize, kSize), groups_of(p.C, kSize)};
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
    const int groups = p.count ? p.pairs / size + (p.pairs < p.E ? p.pairs : p.E) : groups_of(p.C, size);
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

// ---- dgrad ----

constexpr int kGradCols = 64;      // columns of a workgroup

template <int MT> inline constexpr int kSlot = 4096 + MT * 1024;    // 32 rows of weights, 32 values of the rows
template <int MT> inline constexpr int kRing = MT == 4 ? 2 : 3;     // slots of a wavefront

#if defined(__HIP_DEVICE_COMPILE__)

template <int N>
__device__ __forceinline__ void wait_loaded()  // all but the wavefront's last N loads
{
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));    // vmcnt(N)
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ void wait_read()    // the wavefront's LDS reads
{
    __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0)
    asm volatile("" ::: "memory");
}

// In a slot, the 32-byte segment c of weight row r's four is at place c ^ (((r >> 1) & 1) | ((r >> 2) &
// 2)), and 16-byte chunk c of row r's four at place c ^ ((r >> 2) & 3): the lanes that LDS serves
// together then touch all banks.
template <int O, int MT>
__device__ __forceinline__ void few_dgrad_rows(const Group &g, uint8_t *lds)
{
    const auto &p = argument();
    const int lane = lane_now(), wave = uniform(threadIdx.x / kWave), i16 = lane & 15, quarter = lane >> 4;
    const int c0 = blockIdx.x * kGradCols;
    const int steps = (p.k + kStep - 1) / kStep, per = (steps + kWaves - 1) / kWaves;
    const int s0 = wave * per, s1 = min(s0 + per, steps);
    const i32x4 wb = buffer(p.w + (size_t)g.e * p.n * p.k + c0, ((int64_t)p.n * p.k - c0) * 2);
    const i32x4 xb = buffer(p.x + (size_t)g.row0 * p.k, (int64_t)g.n * p.k * 2);
    uint32_t w_off[2];
#pragma unroll
    for (int v = 0; v < 2; ++v)
        w_off[v] = (uint32_t)(lane >> 3) * p.n * 2 + (((lane & 7) ^ ((((lane >> 4) & 1) | v * 2) << 1)) << 4);
    const int chunk = (lane & 3) ^ quarter;
    const uint32_t x_off = ((uint32_t)(lane >> 2) * p.k + chunk * 8) * 2;
    uint8_t *ring = lds + wave * (kRing<MT> * kSlot<MT>);
    // the loads of a step; beyond the wavefront's last one they give 0 as well
    auto load = [&](int slot, int s) {
        const bool some = s < s1;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            load_lds(wb, ring + slot * kSlot<MT> + v * 1024, some ? w_off[v & 1] : kNone,
                     some ? (uint32_t)(s * kStep + v * 8) * p.n * 2 : 0u);
        const uint32_t off = some && s * kStep + chunk * 8 < p.k ? x_off : kNone;
#pragma unroll
        for (int t = 0; t < MT; ++t)
            load_lds(xb, ring + slot * kSlot<MT> + 4096 + t * 1024, off + t * 16 * p.k * 2,
                     some ? (uint32_t)s * (kStep * 2) : 0u);
    };
    constexpr int kLoads = 4 + MT;
    const uint32_t base = (uint32_t)(uintptr_t)(LdsBytes)ring;
    const uint32_t w_at = base + (quarter * 8 + (i16 >> 2)) * 128 + (((i16 >> 3) | ((quarter & 1) << 1)) << 5) +
                          (i16 & 3) * 8;
    const uint32_t x_at = base + 4096 + i16 * 64 + ((quarter ^ (i16 >> 2)) << 4);

    f32x4 acc[4][MT] = {};
#pragma unroll
    for (int i = 0; i < kRing<MT>; ++i) load(i, s0 + i);
    int slot = 0;
    for (int s = s0; s < s1; ++s) {
        wait_loaded<(kRing<MT> - 1) * kLoads>();
        bf16x8 wf[4], xf[MT];
        const uint32_t from = slot * kSlot<MT>;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t at = (w_at ^ (c << 5)) + from;
            wf[c] = read_transposed(at, at + 512);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) xf[t] = *(LdsRows)(uintptr_t)(x_at + from + t * 1024);
        wait_read();
        load(slot, s + kRing<MT>);
        slot = slot + 1 == kRing<MT> ? 0 : slot + 1;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < MT; ++t)
                acc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[c], xf[t], acc[c][t], 0, 0, 0);
    }
    wait_loaded<0>();                          // the rings are free
    __syncthreads();
    f32x4 *meet = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < MT; ++t) meet[((wave * 4 + c) * MT + t) * kWave + lane] = acc[c][t];
    __syncthreads();
    // a lane's four sums are columns quarter * 4 .. of row lane & 15
    for (int q = wave; q < 4 * MT; q += kWaves) {
        const int r = (q % MT) * 16 + i16, c = c0 + (q / MT) * 16 + quarter * 4;
        f32x4 v = meet[q * kWave + lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v += meet[(i * 4 * MT + q) * kWave + lane];
        if (r >= g.n || c >= p.n) continue;
        const size_t row = (size_t)g.row0 + r;
        if constexpr (O == to::kBf16) {
            put_four((uint16_t *)p.out + row * p.n + c, v);
        } else {
            const uint16_t *gu = p.in + row * p.n * 2 + c;
            uint16_t *out = (uint16_t *)p.out + row * p.n * 2 + c;
            f32x4 gate{}, up{}, dg, du;
            add_four(gate, gu);
            add_four(up, gu + p.n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = sigmoid(gate[i]);
                du[i] = v[i] * (gate[i] * s);
                dg[i] = v[i] * up[i] * (s * __builtin_fmaf(gate[i], 1.0f - s, 1.0f));
            }
            put_four(out, dg);
            put_four(out + p.n, du);
        }
    }
}

#endif

template <int O, int MT>
__global__ __launch_bounds__(kThreads) void few_dgrad_kernel(Product p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * kRing<MT> * kSlot<MT>];
    static_assert(sizeof(lds) >= kWaves * 4 * MT * kWave * sizeof(f32x4), "the sums' meeting place");
    constexpr int kSize = kCols * MT;
    for (int group = blockIdx.y;; group += gridDim.y) {
        Group g;
        if (p.count) g = find_group(group, kSize);
        else g = Group{0, group * kSize, min(p.C - group * kSize, kSize), groups_of(p.C, kSize)};
        if (group >= g.of) break;
        few_dgrad_rows<O, MT>(g, lds);
        if (group + (int)gridDim.y >= g.of) break;
        __syncthreads();                       // the meeting place is free again
    }
#else
    (void)p;
#endif
}

template <int O, int MT>
hipError_t launch_dgrad(const Product &p, hipStream_t stream)
{
    const int size = kCols * MT;
    const int groups = p.count ? p.pairs / size + (p.pairs < p.E ? p.pairs : p.E) : groups_of(p.C, size);
    return launch(few_dgrad_kernel<O, MT>, dim3((p.n + kGradCols - 1) / kGradCols, std::min(groups, kMostGroups)),
                  dim3(kThreads), 0, stream, p);
}

template <int O>
hipError_t launch_dgrad_by_rows(const Product &p, hipStream_t stream)
{
    switch (row_tiles(p)) {
    case 1: return launch_dgrad<O, 1>(p, stream);
    case 2: return launch_dgrad<O, 2>(p, stream);
    default: return launch_dgrad<O, 4>(p, stream);
    }
}

// ---- wgrad with few tiles and a long sum ----

// 64 x 64 of an expert's output a workgroup, its rows dealt out to the eight wavefronts; both operands
// lie in LDS as dgrad's weights do.
template <int O>
__global__ __launch_bounds__(kThreads) void few_wgrad_kernel(Product p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * kSquareRing * kSquareSlot];
    static_assert(sizeof(lds) >= kWaves * 16 * kWave * sizeof(f32x4), "the sums' meeting place");
    const int lane = lane_now(), wave = uniform(threadIdx.x / kWave), i16 = lane & 15, quarter = lane >> 4;
    const int across = (p.n + kGradCols - 1) / kGradCols, down = (p.m + kGradCols - 1) / kGradCols;
    const int e = blockIdx.x / (across * down), at = blockIdx.x - e * across * down;
    const int m0 = at / across * kGradCols, c0 = (at - at / across * across) * kGradCols;
    int base = 0, n = 0;
    if (p.pairs > 0) {
        if (p.count) expert_rows(p.count, p.offset, e, p.C, p.rows, base, n);
        else n = p.C;
    }
    base = uniform(base);
    n = uniform(n);
    const int steps = ((uint32_t)n + kStep - 1) / kStep, per = (steps + kWaves - 1) / kWaves;
    const int s0 = wave * per, s1 = min(s0 + per, steps);
    uint32_t x_off[2], w_off[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int chunk = (lane & 7) ^ ((((lane >> 4) & 1) | v * 2) << 1);
        x_off[v] = (uint32_t)(lane >> 3) * p.m * 2 + (chunk << 4);
        w_off[v] = (uint32_t)(lane >> 3) * p.n * 2 + (chunk << 4);
    }
    uint8_t *ring = lds + wave * (kSquareRing * kSquareSlot);
    // the loads of a step; past the expert's rows and the wavefront's last step they give 0
    auto load = [&](int slot, int s) {
        const int left = s < s1 ? n - s * kStep : 0;
        const size_t row = (size_t)base + (left > 0 ? s * kStep : 0);
        const i32x4 xb = buffer(p.x + row * p.m + m0, ((int64_t)left * p.m - m0) * 2);
        const i32x4 wb = buffer(p.w + row * p.n + c0, ((int64_t)left * p.n - c0) * 2);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            load_lds(wb, ring + slot * kSquareSlot + v * 1024, w_off[v & 1], (uint32_t)v * 16 * p.n);
            load_lds(xb, ring + slot * kSquareSlot + 4096 + v * 1024, x_off[v & 1], (uint32_t)v * 16 * p.m);
        }
    };
    const uint32_t at0 = (uint32_t)(uintptr_t)(LdsBytes)ring + (quarter * 8 + (i16 >> 2)) * 128 +
                         (((i16 >> 3) | ((quarter & 1) << 1)) << 5) + (i16 & 3) * 8;

    f32x4 acc[4][4] = {};
#pragma unroll
    for (int i = 0; i < kSquareRing; ++i) load(i, s0 + i);
    int slot = 0;
    for (int s = s0; s < s1; ++s) {
        wait_loaded<(kSquareRing - 1) * 8>();
        bf16x8 wf[4], xf[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t from = (at0 ^ (c << 5)) + slot * kSquareSlot;
            wf[c] = read_transposed(from, from + 512);
            xf[c] = read_transposed(from + 4096, from + 4096 + 512);
        }
        wait_read();
        load(slot, s + kSquareRing);
        slot ^= 1;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                acc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[c], xf[t], acc[c][t], 0, 0, 0);
    }
    wait_loaded<0>();                          // the rings are free
    __syncthreads();
    f32x4 *meet = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < 4; ++t) meet[(wave * 16 + c * 4 + t) * kWave + lane] = acc[c][t];
    __syncthreads();
    for (int q = wave; q < 16; q += kWaves) {
        const int r = m0 + (q & 3) * 16 + i16, c = c0 + (q >> 2) * 16 + quarter * 4;
        f32x4 v = meet[q * kWave + lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v += meet[(i * 16 + q) * kWave + lane];
        if (r >= p.m || c >= p.n) continue;
        const size_t to = ((size_t)e * p.m + r) * p.n + c;
        if constexpr (O == to::kBf16) {
            put_four((uint16_t *)p.out + to, v);
        } else {
            f32x4 *out = reinterpret_cast<f32x4 *>((float *)p.out + to);
            *out = p.accumulate ? *out + v : v;
        }
    }
#else
    (void)p;
#endif
}

// ---- forward with more rows, few tiles and a long sum ----

#if defined(__HIP_DEVICE_COMPILE__)

// 64 rows x 64 columns of the output a workgroup, the sum dealt out to the eight wavefronts: 32 of it at a
// time, 64 bytes of each row, through rings in LDS.
template <int O>
__device__ __forceinline__ void square(const Group &g, uint8_t *lds)
{
    const auto &p = argument();
    const int lane = lane_now(), wave = uniform(threadIdx.x / kWave), i16 = lane & 15, quarter = lane >> 4;
    const int c0 = blockIdx.x * kGradCols;
    const int steps = (p.k + kStep - 1) / kStep, per = (steps + kWaves - 1) / kWaves;
    const int s0 = wave * per, s1 = min(s0 + per, steps);
    const i32x4 wb = buffer(p.w + ((size_t)g.e * p.n + c0) * p.k, (int64_t)(p.n - c0) * p.k * 2);
    const i32x4 xb = buffer(p.x + (size_t)g.row0 * p.k, (int64_t)g.n * p.k * 2);
    const int chunk = (lane & 3) ^ quarter;
    const uint32_t at = ((uint32_t)(lane >> 2) * p.k + chunk * 8) * 2;
    uint8_t *ring = lds + wave * (kSquareRing * kSquareSlot);
    // the loads of a step; beyond the row's end and the wavefront's last step they give 0
    auto load = [&](int slot, int s) {
        const bool some = s < s1;
        const uint32_t off = some && s * kStep + chunk * 8 < p.k ? at : kNone;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t soff = some ? (uint32_t)t * 32 * p.k + (uint32_t)s * (kStep * 2) : 0u;
            load_lds(wb, ring + slot * kSquareSlot + t * 1024, off, soff);
            load_lds(xb, ring + slot * kSquareSlot + 4096 + t * 1024, off, soff);
        }
    };
    const uint32_t from = (uint32_t)(uintptr_t)(LdsBytes)ring + i16 * 64 + ((quarter ^ (i16 >> 2)) << 4);

    f32x4 acc[4][4] = {};
#pragma unroll
    for (int i = 0; i < kSquareRing; ++i) load(i, s0 + i);
    int slot = 0;
    for (int s = s0; s < s1; ++s) {
        wait_loaded<(kSquareRing - 1) * 8>();
        bf16x8 wf[4], xf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            wf[t] = *(LdsRows)(uintptr_t)(from + slot * kSquareSlot + t * 1024);
            xf[t] = *(LdsRows)(uintptr_t)(from + slot * kSquareSlot + 4096 + t * 1024);
        }
        wait_read();
        load(slot, s + kSquareRing);
        slot ^= 1;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                acc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[c], xf[t], acc[c][t], 0, 0, 0);
    }
    wait_loaded<0>();                          // the rings are free
    __syncthreads();
    f32x4 *meet = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < 4; ++t) meet[(wave * 16 + c * 4 + t) * kWave + lane] = acc[c][t];
    __syncthreads();
    for (int q = wave; q < 16; q += kWaves) {
        const int r = (q & 3) * 16 + i16, c = c0 + (q >> 2) * 16 + quarter * 4;
        f32x4 v = meet[q * kWave + lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v += meet[(i * 16 + q) * kWave + lane];
        if (r >= g.n || c >= p.n) continue;
        put_linear<O>(p, (size_t)g.row0 + r, c, v);
    }
}

#endif

template <int O>
__global__ __launch_bounds__(kThreads) void square_kernel(Product p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * kSquareRing * kSquareSlot];
    static_assert(sizeof(lds) >= kWaves * 16 * kWave * sizeof(f32x4), "the sums' meeting place");
    for (int group = blockIdx.y;; group += gridDim.y) {
        Group g;
        if (p.count) g = find_group(group, kGradCols);
        else g = Group{0, group * kGradCols, min(p.C - group * kGradCols, kGradCols), groups_of(p.C, kGradCols)};
        if (group >= g.of) break;
        square<O>(g, lds);
        if (group + (int)gridDim.y >= g.of) break;
        __syncthreads();                       // the meeting place is free again
    }
#else
    (void)p;
#endif
}

template <int O>
hipError_t launch_squares(const Product &p, hipStream_t stream)
{
    const int size = kGradCols;
    const int groups = p.count ? p.pairs / size + (p.pairs < p.E ? p.pairs : p.E) : groups_of(p.C, size);
    return launch(square_kernel<O>, dim3((p.n + kGradCols - 1) / kGradCols, std::min(groups, kMostGroups)),
                  dim3(kThreads), 0, stream, p);
}

}  // namespace

// Experts that rows spread evenly over them reach.
static double experts_reached(const Product &p)
{
    return p.count ? p.E * (1.0 - std::pow(1.0 - 1.0 / p.E, p.pairs)) : 1.0;
}

// The tiles' time in microseconds: a block of 64 of the sum takes 0.65 for 64 rows, a round of 256
// workgroups at a time, and the weights come at `rate` MB/us.
static double tiles_time(const Product &p, double experts, double rate)
{
    const double mean = p.pairs / experts;
    const double rounds = std::ceil(experts * std::ceil(mean / 64) * std::ceil(p.n / 256.0) / 256);
    return std::max(8.0 + rounds * std::ceil(p.k / 64.0) * 0.65, 4.0 + experts * p.n * p.k * 2e-6 / rate);
}

// A square for each CU at most, and more rows than few_rows reads in one go. Measured (the better of tiles
// and few rows, squares), columns x sum: 64 x 4096, 64 rows 22, 13, 2048 rows 24, 13; 512 x 4096, 256 rows
// 23, 13, 2048 rows (256 squares) 44, 28, 4096 rows 45, 52; 4096 x 4096, 32 rows 16, 19, 64 rows 24, 22,
// 256 rows (256) 45, 24, 512 rows 47, 44; 512 x 16384, 2048 rows 150, 95; 8 experts of 512 x 4096, 512 rows
// 47, 24, 1024 rows (160) 43, 26, 2048 rows (288) 44, 44. The sum's length does not enter, though with sums of
// up to 256 the eight wavefronts have few steps or none: kernel times there, 64 to 2048 rows x 64 to 2048, few
// rows 3.5-4.1, squares 4.7-5.9, tiles 7.6-9.5 (a call on its own takes 8 on the host); 512 5.3, 5.8, 11.6;
// 1024 7.3, 6.8, 16.
static bool squares(const Product &p)
{
    const double experts = experts_reached(p), mean = p.pairs / experts;
    // an expert's last square is half empty on average
    const double groups = p.count ? mean / kGradCols + 0.5 : std::ceil(mean / kGradCols);
    return row_tiles(p) == 4 && experts * groups * std::ceil(p.n / (double)kGradCols) <= 256;
}

// Both kernels' times, from what they read, for rows spread evenly over the experts. Few rows: every
// workgroup reads its weights and its rows, at 7.3 TB/s together, and costs 0.0025. Measured (tiles, few
// rows): one matrix of 4096 x 4096, 1 row 42, 9, 64 rows 43, 24, 96 rows 43, 40, 128 rows 43, 46;
// 1024 x 2048, 256 rows 25, 12; 16384 x 4096, 16 rows 62, 39, 64 rows 64, 94; 128 experts of 1536 x 2048,
// 8 rows 25, 12, 64 rows 80, 68, 256 rows 157, 149, 1024 rows 180, 213; of 2048 x 768, 8 rows 13, 9, 32
// rows 20, 27; 16 of 4096 x 4096, 32 rows 109, 73. Where most rows are one expert's the rule does not see it, and
// this kernel reads that expert's weights once for each of its groups: 256 rows of 128 experts of 1536 x 2048
// spread evenly 180, all of one expert 43 (tiles 28).
bool few_rows(const Product &p, bool swiglu)
{
    const double experts = experts_reached(p), mean = p.pairs / experts, k = p.k;
    const double groups = std::ceil(mean / (kCols * row_tiles(p)));
    const double columns = std::ceil(p.n / 16.0) / (swiglu ? 2 : 1);
    const double few = 8.0 + (groups * experts * p.n * k * 2.0 + columns * p.pairs * k * 2.0) / 7.3e6 +
                       experts * groups * columns * 0.0025;
    if (!swiglu && squares(p)) return true;
    return few < tiles_time(p, experts, 4.9);
}

// Both kernels' times again. Few rows: a workgroup a CU, that costs 1.7 and whose row of weights takes 2.2,
// 2.7 or 3.6 ns for 16, 32 or 64 rows of the expert's; the weights come at 5.0 TB/s (tiles 5.2), and at 10
// for an expert's next rows. Measured (tiles, few rows), sum x columns: 4096 x 4096, 1 row 47, 11, 64 rows
// 48, 20, 512 rows 50, 39, 1024 rows 56, 74; 1024 x 2048, 512 rows 18, 10, 2048 rows 21, 30; 16384 x 4096,
// 1 row 169, 36, 512 rows 173, 121, 1024 rows 184, 238; 8 experts of 4096 x 7168, 1 row 48, 15, 8 rows 50,
// 78; 128 of 1536 x 2048, 8 rows 22, 11, 32 rows 33, 35, 256 rows 124, 150; of 2048 x 768, 32 rows 28, 20,
// 128 rows 43, 43.
bool few_dgrad(const Product &p)
{
    const double experts = experts_reached(p), mean = p.pairs / experts;
    const int tiles = row_tiles(p);
    const double groups = std::ceil(mean / (kCols * tiles));
    const double rounds = std::ceil(experts * groups * std::ceil(p.n / (double)kGradCols) / 256);
    const double row = tiles == 1 ? 0.0022 : tiles == 2 ? 0.0027 : 0.0036;
    const double few = std::max(6.3 + rounds * (1.7 + p.k * row),
                                4.0 + experts * p.n * p.k * 2e-6 * (1 / 5.0 + (groups - 1) / 10.0));
    return few < tiles_time(p, experts, 5.2);
}

static int64_t wgrad_squares(const Product &p)
{
    const int64_t across = (p.n + kGradCols - 1) / kGradCols, down = (p.m + kGradCols - 1) / kGradCols;
    return p.E * across * down;
}

// The long sums: at most a square for each CU, and rows enough that the tiles' one wavefront a sum takes
// longer. Measured (tiles, squares), experts of rows x columns, rows of an expert: one of 64 x 64, 512 10,
// 10, 8192 89, 22; of 1024 x 1024 (256 squares), 512 12, 9, 4096 50, 20, 32768 352, 132; 8 of 256 x 512
// (256), 256 10, 14, 512 12, 12, 1024 18, 11, 4096 50, 29; with two squares a CU, one of 2048 x 1024, 4096
// 50, 38, of 4096 x 512 50, 59.
bool few_wgrad(const Product &p)
{
    return wgrad_squares(p) <= 256 && p.pairs / p.E >= 512;
}

hipError_t launch_few_gemm(const Product &p, hipStream_t stream)
{
    if (squares(p)) return launch_squares<to::kBf16>(p, stream);
    return launch_by_rows<to::kBf16>(p, stream);
}

hipError_t launch_few_swiglu(const Product &p, hipStream_t stream)
{
    return launch_by_rows<to::kSwiglu>(p, stream);
}

hipError_t launch_few_linear(const Product &p, hipStream_t stream)
{
    if (squares(p)) return launch_squares<to::kLinear>(p, stream);
    return launch_by_rows<to::kLinear>(p, stream);
}

hipError_t launch_few_dgrad(const Product &p, bool swiglu, hipStream_t stream)
{
    return swiglu ? launch_dgrad_by_rows<to::kSwigluGrad>(p, stream)
                  : launch_dgrad_by_rows<to::kBf16>(p, stream);
}

hipError_t launch_few_wgrad(const Product &p, bool f32, hipStream_t stream)
{
    return launch(f32 ? few_wgrad_kernel<to::kF32> : few_wgrad_kernel<to::kBf16>, dim3((unsigned)wgrad_squares(p)),
                  dim3(kThreads), 0, stream, p);
}

}  // namespace ep
