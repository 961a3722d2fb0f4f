// The experts' FP8 products on gfx950: each expert's rows (E4M3 codes with one fp32 scale per row
// and 128 channels, as the FP8 dispatch writes them) times its weights (E4M3 codes with one fp32
// scale per 128 x 128 block).
//
//   y[r][c] = bf16( sum_b xs[r][b] * ws[e][c / 128][b] * sum_{k in block b} xq[r][k] * wq[e][c][k] )
//
// One v_mfma_f32_16x16x128_f8f6f4 covers exactly one scale block of a 16 x 16 tile, so the inner
// sum is one matrix instruction with a zero start and the outer sum one fmaf per element, in
// ascending b. The SwiGLU form, whose scales are fp32 outputs, takes the exact product of the same
// codes (mfma_exact). The weights are the A operand and the rows the B operand: a lane then holds one
// row (its scale is one value) and four consecutive output channels.
#include "ep_expert.h"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kTileN = 256;        // weight rows per workgroup: 64 per wavefront

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The experts' rows cut into tiles of `bm` rows: rows and first row of each expert, and the
// running number of tiles. Built once per workgroup.
struct TileTable {
    int32_t end[EP_MAX_EXPERTS], base[EP_MAX_EXPERTS], n[EP_MAX_EXPERTS];
    int32_t wave_sum[16];
};

template <int THREADS>
__device__ __forceinline__ int build_table(TileTable &t, const ExpertProduct &p, int bm)
{
    constexpr int kPer = EP_MAX_EXPERTS / THREADS;
    const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
    const int e0 = threadIdx.x * kPer;
    int tiles[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        tiles[i] = 0;
        if (e0 + i < p.E) {
            int base, n;
            expert_rows(p.count, p.offset, e0 + i, p.C, p.rows, base, n);
            t.base[e0 + i] = base;
            t.n[e0 + i] = n;
            tiles[i] = (n + bm - 1) / bm;
        }
        sum += tiles[i];
    }
    const int incl = wave_inclusive_sum(sum);
    if (lane == kWave - 1) t.wave_sum[wave] = incl;
    __syncthreads();
    int run = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) {
        const int s = t.wave_sum[w];
        if (w < wave) run += s;
        total += s;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        run += tiles[i];
        if (e0 + i < p.E) t.end[e0 + i] = run;
    }
    __syncthreads();
    return total;
}

// The tiles of all experts in one row, an expert's tiles in groups of kGroup row tiles: within a
// group the row tile runs fastest, then the column tile. Neighbours in this order share weights
// and rows, and each XCD takes one eighth of the order (its workgroups are blockIdx.x mod 8), so
// that its L2 holds what they share.
constexpr int kGroup = 8;

struct TileRange {
    int first, end, step;
};

__device__ __forceinline__ TileRange my_tiles(int total)
{
    const int x = blockIdx.x & 7, i = blockIdx.x >> 3;      // gridDim.x is a multiple of 8
    const int per = total >> 3, rest = total & 7;
    const int first = x * per + min(x, rest);
    return TileRange{first + i, first + per + (x < rest ? 1 : 0), (int)(gridDim.x >> 3)};
}

struct Tile {
    int e, row0, n, nblk;      // expert, first row, rows, column tile
};

// The tile at place `tile` of the order (below the total); lanes may ask for different ones.
__device__ __forceinline__ Tile locate(const TileTable &t, int E, int tile, int n_tiles, int bm)
{
    const int m = tile / n_tiles;
    int lo = 0, hi = E - 1;    // the expert whose row tiles include m
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.end[mid] > m) hi = mid;
        else lo = mid + 1;
    }
    const int n_e = t.n[lo], tiles = (n_e + bm - 1) / bm;
    int at = tile - (t.end[lo] - tiles) * n_tiles;
    const int group = at / (kGroup * n_tiles), in_group = min(tiles - group * kGroup, kGroup);
    at -= group * kGroup * n_tiles;
    Tile r;
    r.e = lo;
    r.nblk = at / in_group;
    const int m0 = (group * kGroup + at - r.nblk * in_group) * bm;
    r.row0 = t.base[lo] + m0;
    r.n = min(n_e - m0, bm);
    return r;
}

__device__ __forceinline__ Tile uniform(const Tile &t)
{
    return Tile{uniform(t.e), uniform(t.row0), uniform(t.n), uniform(t.nblk)};
}

// h = silu(g) * u; the reciprocal is the hardware's (one step of fp32). g = -inf gives NaN, as
// -inf / inf does.
__device__ __forceinline__ float swiglu(float g, float u)
{
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// The scale of a block with this amax pattern (integer max of |h|): amax / 448, a NaN amax giving
// the quiet NaN (the rules of the FP8 dispatch).
__device__ __forceinline__ float block_scale(uint32_t amax)
{
    return amax > 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(amax) / 448.0f;
}

// E4M3 codes of four values of a block: q = e4m3(h / scale), IEEE division; signed zeros where
// the scale is 0, and every code carries its value's own sign.
__device__ __forceinline__ uint32_t encode4_any(const float (&h)[4], float scale)
{
    uint32_t v = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t sign = (__float_as_uint(h[k]) >> 24) & 0x80u;
        const uint32_t c = scale == 0.0f ? sign : sign | (e4m3_rne_sat(h[k] / scale) & 0x7Fu);
        v |= c << (8 * k);
    }
    return v;
}

// bf16 pairs of four values, NaN as 0x7FC0.
__device__ __forceinline__ uint2 bf16_pairs(float a, float b, float c, float d)
{
    const float v[4] = {a, b, c, d};
    bf16x2 lo = {(__bf16)v[0], (__bf16)v[1]}, hi = {(__bf16)v[2], (__bf16)v[3]};
    uint2 o{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    if (__builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3])) {
        o.x = bf16_rne(v[0]) | (bf16_rne(v[1]) << 16);
        o.y = bf16_rne(v[2]) | (bf16_rne(v[3]) << 16);
    }
    return o;
}

// The SwiGLU epilogue of one tile of ROWS rows x 128 channels of h: the block amax meets in LDS, the
// codes go out through LDS in whole rows. A wavefront holds quarter `part` of the 128 channels, a
// lane G groups of 4 consecutive ones (group g at channel part * 32 + channel(g)) of M rows
// (row(m)), GROUP lanes apart from the other channels of the row; one that holds none only helps
// to store.
template <int ROWS>
struct SwigluShared {
    uint32_t amax[4][ROWS];
    float scale[ROWS];
    u32x4 code[ROWS][8];
};

template <int THREADS, int ROWS, int M, int G, int GROUP, typename Row, typename Channel>
__device__ __forceinline__ void store_swiglu(SwigluShared<ROWS> &sh, float (&h)[M][G][4],
                                             bool holds, int part, Row row, Channel channel, const ExpertProduct &p,
                                             int row0, int n, int nblk)
{
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        uint32_t amax = 0;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                amax = max(amax, __float_as_uint(h[m][g][k]) & 0x7FFFFFFFu);
#pragma unroll
        for (int x = GROUP; x < kWave; x *= 2) amax = max(amax, (uint32_t)__shfl_xor((int)amax, x));
        if (holds && lane < GROUP) sh.amax[part][row(m)] = amax;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if (!holds) break;
        const int r = row(m);
        uint32_t amax = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) amax = max(amax, sh.amax[w][r]);
        const float scale = block_scale(amax);
        // 2^-60 <= amax < inf: the quotients lie where div_by_rcp and the conversion are exact
        const bool plain = __any(amax < 0x21800000u || amax >= 0x7F800000u);
        const float y = 1.0f / scale;
        uint32_t *code = reinterpret_cast<uint32_t *>(&sh.code[r][0]) + part * 8;
        if (plain) {
#pragma unroll 1
            for (int g = 0; g < G; ++g) {
                float v[4];                    // h[m][g] by selects: g is not constant here
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = h[m][0][k];
#pragma unroll
                    for (int i = 1; i < G; ++i) v[k] = i == g ? h[m][i][k] : v[k];
                }
                code[channel(g) >> 2] = encode4_any(v, scale);
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g)
                code[channel(g) >> 2] =
                    e4m3_pack4(div_by_rcp(h[m][g][0], scale, y), div_by_rcp(h[m][g][1], scale, y),
                               div_by_rcp(h[m][g][2], scale, y), div_by_rcp(h[m][g][3], scale, y));
        }
        if (part == 0 && lane < GROUP) sh.scale[r] = scale;
    }
    __syncthreads();
    const int I = p.n / 2;
    for (int i = threadIdx.x; i < ROWS * 8; i += THREADS) {
        const int r = i >> 3;
        if (r < n)
            *reinterpret_cast<u32x4 *>(p.h_q + (size_t)(row0 + r) * I + nblk * 128 + (i & 7) * 16) =
                sh.code[r][i & 7];
    }
    for (int r = threadIdx.x; r < n; r += THREADS)
        p.h_scale[(size_t)(row0 + r) * (I / 128) + nblk] = sh.scale[r];
    __syncthreads();
}

// Few rows per expert, where reading the weights bounds the product: every operand straight from
// global memory to registers, no barrier in the product. MT tiles of 16 rows; a wavefront takes 4
// tiles of 16 weight rows (gemm: 64 consecutive rows; SwiGLU: 32 gate rows and the same 32 up rows),
// D blocks in flight. KS wavefronts share the same weight rows, each every KS-th block, and their
// sums meet in LDS in order: with few tiles that keeps more of the chip's memory busy.
template <int MT, bool SWIGLU, int D, int KS>
__global__ __launch_bounds__(kThreads *KS) void expert_stream_kernel(ExpertProduct p)
{
    constexpr int kStreamThreads = kThreads * KS;
    __shared__ TileTable table;
    __shared__ SwigluShared<SWIGLU ? MT * 16 : 1> sh;
    __shared__ f32x4 parts[KS > 1 ? KS - 1 : 1][KS > 1 ? 4 : 1][KS > 1 ? 4 * MT : 1][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave) & 3, ks = uniform(threadIdx.x / kThreads);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int nkb = p.H >> 7;
    const int n_tiles = SWIGLU ? p.n / kTileN : (p.n + kTileN - 1) / kTileN;
    const int ws_rows = (p.n + 127) >> 7;
    const int total = build_table<kStreamThreads>(table, p, MT * 16) * n_tiles;
    const TileRange mine = my_tiles(total);
    for (int tile = mine.first; tile < mine.end; tile += mine.step) {
        const Tile at = uniform(locate(table, p.E, tile, n_tiles, MT * 16));
        const int e = at.e, row0 = at.row0, n = at.n, nblk = at.nblk;

        // lane offsets of the weight rows (clamped) and of the tile's rows (clamped)
        uint32_t woff[4], xoff[MT], soff[MT];
        int wrow[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            wrow[nt] = SWIGLU ? (nt >> 1) * (p.n / 2) + nblk * 128 + wave * 32 + (nt & 1) * 16
                              : nblk * kTileN + wave * 64 + nt * 16;
            woff[nt] = (uint32_t)min(wrow[nt] + r16, p.n - 1) * p.H + g4 * 16;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = min(mt * 16 + r16, n - 1);
            xoff[mt] = (uint32_t)r * p.H + g4 * 16;
            soff[mt] = (uint32_t)r * nkb;
        }
        const uint8_t *w = p.w_q + (size_t)e * p.n * p.H;
        const uint8_t *x = p.q + (size_t)row0 * p.H;
        const float *xs = p.scale + (size_t)row0 * nkb;
        const float *ws[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            ws[i] = p.w_scale + ((size_t)e * ws_rows + min(wrow[2 * i] >> 7, ws_rows - 1)) * nkb;

        i32x8 wf[D][4], xf[D][MT];
        float sx[D][MT], sw[D][2];
        auto load = [&](int d, int kb) {
            const uint8_t *wk = w + kb * 128, *xk = x + kb * 128;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
                wf[d][nt] = join(*reinterpret_cast<const i32x4 *>(wk + woff[nt]),
                                 *reinterpret_cast<const i32x4 *>(wk + woff[nt] + 64));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                xf[d][mt] = join(*reinterpret_cast<const i32x4 *>(xk + xoff[mt]),
                                 *reinterpret_cast<const i32x4 *>(xk + xoff[mt] + 64));
                sx[d][mt] = xs[kb + soff[mt]];
            }
            sw[d][0] = ws[0][kb];
            sw[d][1] = ws[1][kb];
        };
        f32x4 acc[4][MT];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[nt][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (ks < nkb) {
#pragma unroll
            for (int d = 0; d < D; ++d) load(d, min(ks + d * KS, nkb - 1));
            for (int kb = ks; kb < nkb; kb += D * KS) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (kb + d * KS < nkb) {
                        Bf16Block xb[SWIGLU ? MT : 1];
                        if constexpr (SWIGLU)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) xb[mt] = bf16_block(xf[d][mt]);
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt) {
                            Bf16Block wb;
                            if constexpr (SWIGLU) wb = bf16_block(wf[d][nt]);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                f32x4 v;
                                if constexpr (SWIGLU) v = mfma_exact(wb, xb[mt]);
                                else v = mfma_e4m3(wf[d][nt], xf[d][mt]);
                                const float s = sx[d][mt] * sw[d][nt >> 1];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    acc[nt][mt][k] = __builtin_fmaf(s, v[k], acc[nt][mt][k]);
                            }
                        }
                    }
                    load(d, min(kb + (d + D) * KS, nkb - 1));
                }
            }
        }
        if constexpr (KS > 1) {
            if (ks > 0)
#pragma unroll
                for (int i = 0; i < 4 * MT; ++i) parts[ks - 1][wave][i][lane] = acc[i / MT][i % MT];
            __syncthreads();
            if (ks == 0)
#pragma unroll
                for (int i = 0; i < 4 * MT; ++i)
#pragma unroll
                    for (int j = 0; j < KS - 1; ++j) acc[i / MT][i % MT] += parts[j][wave][i][lane];
            __syncthreads();
        }

        if constexpr (SWIGLU) {
            float h[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[mt][g][k] = swiglu(acc[g][mt][k], acc[g + 2][mt][k]);
            store_swiglu<kStreamThreads, MT * 16, MT, 2, 16>(
                sh, h, ks == 0, wave, [&](int m) { return m * 16 + r16; },
                [&](int g) { return g * 16 + g4 * 4; }, p, row0, n, nblk);
        } else if (ks == 0) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int r = mt * 16 + r16;
                uint16_t *y = p.y + (size_t)(row0 + r) * p.n;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const int c = wrow[nt] + g4 * 4;
                    // n % 8 == 0: the four channels together
                    if (r < n && c < p.n)
                        *reinterpret_cast<uint2 *>(y + c) = bf16_pairs(
                            acc[nt][mt][0], acc[nt][mt][1], acc[nt][mt][2], acc[nt][mt][3]);
                }
            }
        }
    }
}

// Many rows per expert: tiles of 128 rows x 256 weight rows (SwiGLU: 128 gate and the same 128 up
// rows), one workgroup of 8 wavefronts per CU that walks its tiles as one stream of blocks (128
// channels of a tile each); a wavefront multiplies 64 rows by 64 weight rows. Two wavefronts per
// SIMD share its issue slots: alone, a wavefront's scaled sums, LDS reads and products queue up. Loads run two blocks ahead of LDS and three ahead of the products,
// across tiles, so that neither a block nor a tile waits for memory. A load instruction covers 8
// whole 128-byte row segments, 8 lanes a row: the vector cache takes one access per 128 bytes (in
// the matrix instruction's lane order, 16 rows side by side, it took one per 16 bytes, and that
// bounded the kernel: 1.35 ms for 65536 rows x 4096 x 4096). From registers a block goes to one of
// two LDS buffers, an eighth per wavefront. The row scales of 16 blocks are staged together, one
// panel ahead. One barrier per block.
constexpr int kTileThreads = 512;
constexpr int kTileM = 128;
[[maybe_unused]] constexpr int kMT = 2;     // tiles of 32 rows of a wavefront
constexpr int kPanel = 16;         // blocks whose scales are staged together
constexpr int kList = 256;         // tiles of a workgroup looked up together

// A buffer of `bytes` from p: loads take a lane offset and a uniform one, and give 0 past the end.
[[maybe_unused]] __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00027000);
}

[[maybe_unused]] __device__ __forceinline__ i32x4 buffer_load16(__amdgpu_buffer_rsrc_t b, int lane_off, int off)
{
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_off, off, 0));
}

// v, but what is computed from it is worked out where it is used and not kept in registers.
[[maybe_unused]] __device__ __forceinline__ int fresh(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// Meet the other wavefronts with LDS settled; loads in flight stay in flight.
[[maybe_unused]] __device__ __forceinline__ void meet()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <bool SWIGLU>
struct TileShared {
    u32x4 x[2][kTileM * 8];
    u32x4 w[2][kTileN * 8];
    float xscale[2][kPanel][kTileM + 1];
    float wscale[2][kPanel][2];
    int4 list[kList];
    SwigluShared<SWIGLU ? kTileM : 1> h;
};

template <bool SWIGLU>
__global__ __launch_bounds__(kTileThreads) void expert_tile_kernel(ExpertProduct p)
{
#if defined(__HIP_DEVICE_COMPILE__)            // buffer descriptors exist on the device only
    __shared__ TileTable table;
    __shared__ TileShared<SWIGLU> sh;
    const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
    const int wm = wave & 1, wn = wave >> 1;   // the wavefront's 64 rows and its weight rows
    const int r32 = lane & 31, half = lane >> 5;
    const int nkb = p.H >> 7;
    const int n_tiles = (p.n + kTileN - 1) / kTileN;
    const int ws_rows = (p.n + 127) >> 7;
    const int total = build_table<kTileThreads>(table, p, kTileM) * n_tiles;
    const TileRange mine = my_tiles(total);
    // Chunk c (16 bytes) of row r is kept at place c ^ swizzle(r) of the row's eight: the lanes that
    // LDS serves together (8 consecutive rows, and the same 16 further on) then touch all banks.
    // A lane's j-th chunk of a block is 2 * j + half of row lane & 31.
    auto swizzle = [](int r) { return (r & 7) ^ ((r >> 4) & 1); };
    const int row_at = r32 * 8, row_swizzle = swizzle(r32);

    // the stream of loads: the tile it is in and its next block
    struct {
        int tile, kb;
        __amdgpu_buffer_rsrc_t w, x;
        int woff[4], xoff[2];
    } ld;
    // Weight row i of a tile: SwiGLU keeps 32 gate rows and the same 32 up rows together, so that
    // every wavefront has a tile of each.
    auto weight_row = [&](int nblk, int i) {
        return SWIGLU ? ((i >> 5) & 1) * (p.n / 2) + nblk * 128 + (i >> 6) * 32 + (i & 31)
                      : nblk * kTileN + i;
    };
    auto at = [&](int i) {
        const int4 v = sh.list[i];
        return uniform(Tile{v.x, v.y, v.z, v.w});
    };
    auto enter = [&](int i) {
        const Tile t = at(i);
        ld.tile = i;
        ld.kb = 0;
        ld.w = buffer(p.w_q + (size_t)t.e * p.n * p.H, (uint32_t)p.n * p.H);
        ld.x = buffer(p.q + (size_t)t.row0 * p.H, (uint32_t)t.n * p.H);
        const int l = fresh(lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ld.woff[j] = min(weight_row(t.nblk, wave * 32 + j * 8 + (l >> 3)), p.n - 1) * p.H +
                         (l & 7) * 16;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            ld.xoff[j] = min(wave * 16 + j * 8 + (l >> 3), t.n - 1) * p.H + (l & 7) * 16;
    };

    constexpr int kStage = SWIGLU ? 1 : 2;     // blocks in registers on their way to LDS
    i32x4 wr[kStage][4], xr[kStage][2];
    i32x4 wf[2][4];                            // the wavefront's weights of a block: [tile][chunk]
    f32x16 acc[2][kMT];
    constexpr int kXf = SWIGLU ? 1 : 2;
    i32x4 xf[kXf][4];
    constexpr int kWs = SWIGLU ? 2 : 1;
    float xs[2];                               // row scales
    constexpr int kPer = kTileM * kPanel / kTileThreads;
    float ps[kPer], pw = 0.0f;                 // the next panel on its way
    int par = 0;                               // the panel in use

    auto load_w = [&](int d, int j) { wr[d % kStage][j] = buffer_load16(ld.w, ld.woff[j], ld.kb * 128); };
    auto load_x = [&](int d, int j) { xr[d % kStage][j] = buffer_load16(ld.x, ld.xoff[j], ld.kb * 128); };
    // the lane's place in LDS: its row of each 8, its chunk (rows 16 further on swap neighbours)
    const int put0 = (lane >> 3) * 8 + ((lane & 7) ^ (lane >> 3));
    auto put_w = [&](int d, int j) {
        sh.w[d][wave * 256 + j * 64 + (put0 ^ (j >> 1))] = __builtin_bit_cast(u32x4, wr[d % kStage][j]);
    };
    auto put_x = [&](int d, int j) {
        sh.x[d][wave * 128 + j * 64 + (put0 ^ (wave & 1))] = __builtin_bit_cast(u32x4, xr[d % kStage][j]);
    };
    auto advance = [&](int tiles) {            // past the last block: that block again
        if (++ld.kb == nkb) {
            if (ld.tile + 1 < tiles) enter(ld.tile + 1);
            else ld.kb = nkb - 1;
        }
    };
    auto panel_load = [&](int i, int kb0) {
        const Tile t = at(i);
        const int l = fresh(wave * kWave + lane);
        const float *src = p.scale + (size_t)t.row0 * nkb + min(kb0 + (l & 15), nkb - 1);
#pragma unroll
        for (int k = 0; k < kPer; ++k) ps[k] = src[(size_t)min(k * 32 + (l >> 4), t.n - 1) * nkb];
        const int blk = SWIGLU ? ((l >> 4) & 1) * (p.n >> 8) + t.nblk
                               : min(t.nblk * 2 + ((l >> 4) & 1), ws_rows - 1);
        pw = p.w_scale[((size_t)t.e * ws_rows + blk) * nkb + min(kb0 + (l & 15), nkb - 1)];
    };
    auto panel_store = [&](int to) {
        const int l = fresh(wave * kWave + lane);
#pragma unroll
        for (int k = 0; k < kPer; ++k) sh.xscale[to][l & 15][k * 32 + (l >> 4)] = ps[k];
        if (l < 32) sh.wscale[to][l & 15][l >> 4] = pw;
    };
    auto read_row = [&](int d, int mt) {       // the lane's chunks of row tile mt
        const i32x4 *x = reinterpret_cast<const i32x4 *>(sh.x[d]) + (wm * kMT + mt) * 256 + row_at;
#pragma unroll
        for (int j = 0; j < 4; ++j) xf[mt % kXf][j] = x[(2 * j + half) ^ row_swizzle];
    };
    auto read_w = [&](int d, int nt) {         // and of the wavefront's weight tile nt
        const i32x4 *w = reinterpret_cast<const i32x4 *>(sh.w[d]) + (wn * 2 + nt) * 256 + row_at;
#pragma unroll
        for (int j = 0; j < 4; ++j) wf[nt][j] = w[(2 * j + half) ^ row_swizzle];
    };
    float ws[kWs];
    auto read_ws = [&](float (&to)[kWs], int b) {
        to[0] = sh.wscale[par][b][SWIGLU ? 0 : wn >> 1];
        if constexpr (SWIGLU) to[1] = sh.wscale[par][b][1];
    };
    auto clear = [&]() {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[nt][mt][i] = 0.0f;
    };
    // One block, in LDS buffer d, in 2 regions of one tile of 32 rows each, kept apart by fences. The
    // next block goes to LDS before the barrier, and the one three ahead takes its registers.
    auto step = [&](int d, int tile, int kb, int tiles) {
        const int dn = d ^ 1;
        if ((kb & (kPanel - 1)) == 0) {
            if (kb + kPanel < nkb) panel_load(tile, kb + kPanel);
            else if (tile + 1 < tiles) panel_load(tile + 1, 0);
        }
        const int b_next = kb == nkb - 1 ? 0 : (kb + 1) & (kPanel - 1);
        float ws_next[kWs];
        bf16x8 wb[SWIGLU ? 2 : 1][8];
        read_w(d, 0);
        read_w(d, 1);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            // the row tile to read: SwiGLU, short of registers, this one; else the one after, the
            // last of them the next block's
            const int to = SWIGLU ? mt : mt + 1;
            if constexpr (SWIGLU) {
                read_row(d, mt);
                xs[mt] = sh.xscale[par][kb & (kPanel - 1)][(wm * kMT + mt) * 32 + r32];
            }
            if (mt == kMT - 1) {
                if (b_next == 0) {
                    par ^= 1;
                    panel_store(par);
                }
                meet();
                read_ws(ws_next, b_next);
            }
            if constexpr (!SWIGLU) {
                read_row(to < kMT ? d : dn, to & (kMT - 1));
                xs[to & 1] = sh.xscale[par][to < kMT ? kb & (kPanel - 1) : b_next]
                                      [(wm * kMT + (to & (kMT - 1))) * 32 + r32];
            }
            if (mt < kMT - 1) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    put_x(dn, j);
                    load_x(dn, j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    put_w(dn, j);
                    load_w(dn, j);
                }
            }
            f32x16 v[2] = {};
            if constexpr (SWIGLU) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bf16x8 xb = bf16_of_e4m3(xf[0][j >> 1][(j & 1) * 2],
                                                   xf[0][j >> 1][(j & 1) * 2 + 1]);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        if (mt == 0)
                            wb[nt][j] = bf16_of_e4m3(wf[nt][j >> 1][(j & 1) * 2],
                                                     wf[nt][j >> 1][(j & 1) * 2 + 1]);
                        v[nt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[nt][j], xb, v[nt], 0, 0,
                                                                        0);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
                        v[nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            join(wf[nt][2 * j], wf[nt][2 * j + 1]),
                            join(xf[mt % kXf][2 * j], xf[mt % kXf][2 * j + 1]), v[nt], 0, 0, 0, 0, 0,
                            0);
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const float s = xs[mt & 1] * ws[SWIGLU ? nt : 0];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[nt][mt][i] = __builtin_fmaf(s, v[nt][i], acc[nt][mt][i]);
                asm volatile("" : "+v"(acc[nt][mt]));    // summed here, not later
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < kWs; ++i) ws[i] = ws_next[i];
        advance(tiles);
    };
    auto finish = [&](int tile) {              // the tile's output
        const Tile t = at(tile);
        const int l = fresh(lane);
        // element i of a lane is channel (i >> 2) * 8 + half * 4 + (i & 3) of row lane & 31
        if constexpr (SWIGLU) {
            float h[kMT][4][4];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int i = 0; i < 16; ++i) h[mt][i >> 2][i & 3] = swiglu(acc[0][mt][i], acc[1][mt][i]);
            store_swiglu<kTileThreads, kTileM, kMT, 4, 32>(
                sh.h, h, true, wn, [&](int m) { return (wm * kMT + m) * 32 + (l & 31); },
                [&](int g) { return g * 8 + (l >> 5) * 4; }, p, t.row0, t.n, t.nblk);
        } else {
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
                const int r = (wm * kMT + mt) * 32 + (l & 31);
                uint16_t *y = p.y + (size_t)(t.row0 + r) * p.n;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int c = weight_row(t.nblk, wn * 64 + nt * 32) + g * 8 + (l >> 5) * 4;
                        // n % 8 == 0: the four channels together
                        if (r < t.n && c < p.n)
                            *reinterpret_cast<uint2 *>(y + c) =
                                bf16_pairs(acc[nt][mt][g * 4], acc[nt][mt][g * 4 + 1],
                                           acc[nt][mt][g * 4 + 2], acc[nt][mt][g * 4 + 3]);
                    }
            }
        }
        clear();
    };

#pragma unroll
    for (int k = 0; k < kPer; ++k) ps[k] = 0.0f;
    for (int first = mine.first; first < mine.end; first += kList * mine.step) {
        const int tiles = min((mine.end - first + mine.step - 1) / mine.step, kList);
        if ((int)threadIdx.x < tiles) {
            const int i = fresh(threadIdx.x);
            const Tile t = locate(table, p.E, first + i * mine.step, fresh(n_tiles), kTileM);
            sh.list[threadIdx.x] = int4{t.e, t.row0, t.n, t.nblk};
        }
        __syncthreads();
        enter(0);
        par = 0;
        panel_load(0, 0);
        auto load = [&](int d) {
#pragma unroll
            for (int j = 0; j < 2; ++j) load_x(d, j);
#pragma unroll
            for (int j = 0; j < 4; ++j) load_w(d, j);
            advance(tiles);
        };
        load(0);
        if constexpr (kStage == 2) load(1);
        panel_store(0);
#pragma unroll
        for (int j = 0; j < 2; ++j) put_x(0, j);
#pragma unroll
        for (int j = 0; j < 4; ++j) put_w(0, j);
        load(0);
        meet();
        read_ws(ws, 0);
        clear();
        if constexpr (!SWIGLU) read_row(0, 0);
        xs[0] = sh.xscale[0][0][wm * kMT * 32 + r32];
        __builtin_amdgcn_sched_barrier(0);
        int tile = 0, kb = 0;
        auto next = [&](int d) {               // a block; false after the last one
            step(d, tile, kb, tiles);
            if (++kb < nkb) return true;
            finish(tile);
            kb = 0;
            return ++tile < tiles;
        };
        while (next(0) && next(1)) {}
        meet();                                // the list and LDS are free again
    }
#else
    (void)p;
#endif
}

#ifndef EP_EXPERT_MT1
#define EP_EXPERT_MT1 12
#endif
#ifndef EP_EXPERT_MT2
#define EP_EXPERT_MT2 24
#endif
#ifndef EP_EXPERT_TILE
#define EP_EXPERT_TILE 40
#endif
#ifndef EP_EXPERT_KS
#define EP_EXPERT_KS 512
#endif
#ifndef EP_EXPERT_D1
#define EP_EXPERT_D1 1
#endif
template <bool SWIGLU>
hipError_t launch_product(const ExpertProduct &p, hipStream_t stream)
{
    if (p.pairs == 0 || (p.offset && p.rows == 0)) return hipSuccess;
    const int64_t n_tiles = (p.n + kTileN - 1) / kTileN;
    const int mean = (int)(((int64_t)p.pairs + p.E - 1) / p.E);
    // the grid: at most `most` workgroups, no more than there can be tiles of `bm` rows
    auto grid = [&](int bm, int64_t most) {
        const int64_t experts = p.pairs < p.E ? p.pairs : p.E;
        const int64_t tiles = (p.pairs / bm + experts) * n_tiles;
        return dim3((unsigned)(tiles < most ? (tiles + 7) / 8 * 8 : most));
    };
    const dim3 block(kThreads);
    if (mean >= EP_EXPERT_TILE)
        return launch(expert_tile_kernel<SWIGLU>, grid(kTileM, 256), dim3(kTileThreads), 0, stream, p);
    if (mean > EP_EXPERT_MT2)
        return launch(expert_stream_kernel<4, SWIGLU, 1, 1>, grid(64, 512), block, 0, stream, p);
    if (mean > EP_EXPERT_MT1)
        return launch(expert_stream_kernel<2, SWIGLU, 1, 1>, grid(32, 512), block, 0, stream, p);
    if (grid(16, 1 << 20).x < EP_EXPERT_KS)
        return launch(expert_stream_kernel<1, SWIGLU, 1, 4>, grid(16, 512), dim3(4 * kThreads), 0,
                      stream, p);
    return launch(expert_stream_kernel<1, SWIGLU, EP_EXPERT_D1, 1>, grid(16, 1024), block, 0, stream, p);
}

}  // namespace

hipError_t launch_expert_gemm_fp8(const ExpertProduct &p, hipStream_t stream)
{
    return launch_product<false>(p, stream);
}

hipError_t launch_expert_swiglu_fp8(const ExpertProduct &p, hipStream_t stream)
{
    return launch_product<true>(p, stream);
}

}  // namespace ep
