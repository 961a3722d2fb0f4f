// The experts' FP8 products on gfx950: each expert's rows (E4M3 codes with one fp32 scale per row
// and 128 channels, as the FP8 dispatch writes them) times its weights (E4M3 codes with one fp32
// scale per 128 x 128 block).
//
//   y[r][c] = bf16( sum_b xs[r][b] * ws[e][c / 128][b] * sum_{k in block b} xq[r][k] * wq[e][c][k] )
//
// The inner sum of a 32 x 32 tile is two matrix instructions of 64 channels with a zero start, the
// outer sum one fmaf per element, in ascending b. The SwiGLU form, whose scales are fp32 outputs,
// takes the exact product of the same codes, as bf16 (bf16_of_e4m3). The weights are the A operand
// and the rows the B operand: a lane then holds one row (its scale is one value) and groups of four
// consecutive output channels.
#include "ep_expert.h"

#include <type_traits>

namespace ep {

namespace {

constexpr int kTileThreads = 512;
constexpr int kTileN = 256;        // weight rows of a tile
template <int MT> inline constexpr int kTileRows = 64 * MT;     // rows of a tile

#if defined(__HIP_DEVICE_COMPILE__)            // buffer descriptors exist on the device only

using ep::uniform;                  // the form for a Tile, below, would hide it

// The lane, counted anew: what is computed from it is worked out where it is used, and takes no
// register through the product (which needs them all).
__device__ __forceinline__ int lane_now()
{
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
    return l;
}

// The experts' rows cut into tiles of `bm` rows: rows and first row of each expert, and the
// running number of tiles. Built once per workgroup.
struct TileTable {
    int32_t end[EP_MAX_EXPERTS], base[EP_MAX_EXPERTS], n[EP_MAX_EXPERTS];
    int32_t wave_sum[2][kTileThreads / kWave];
};

struct Tiling {
    int total, mt;                 // row tiles of all experts, of 64 * mt rows
};

// Builds the table and chooses the height of the tiles from the rows there are. A workgroup takes 1.35
// to 1.5 times as long for a tile of 128 rows as for one of 64 (the weights' share of the loads and
// LDS reads is the same): 19.4 against 14.6 us with one tile each of 4 experts' rows, 39.5 for two
// against 41.1 for three, H = 2048; SwiGLU 30.3 against 21.7 us, and 64.5 against 63.6. So the taller
// tiles pay where they leave less than 5/7 as many tiles for the busiest workgroup. Few rows an
// expert, or few tiles: 64 rows (8 rows for each of 128 experts, gate/up of 2 x 768 x 2048, 79 us
// against 111); more: 128 rows (341 rows for each of 96 experts, 250 us against 302).
__device__ __forceinline__ Tiling build_table(TileTable &t, const ExpertProduct &p, int n_tiles)
{
    constexpr int kPer = EP_MAX_EXPERTS / kTileThreads, kWaves = kTileThreads / kWave;
    const int lane = lane_now(), wave = uniform(threadIdx.x / kWave);
    const int e0 = (wave * kWave + lane) * kPer;
    int tiles[2][kPer], sum[2] = {0, 0}, incl[2];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        tiles[0][i] = tiles[1][i] = 0;
        if (e0 + i < p.E) {
            int base, n;
            expert_rows(p.count, p.offset, e0 + i, p.C, p.rows, base, n);
            t.base[e0 + i] = base;
            t.n[e0 + i] = n;
            tiles[0][i] = (n + kTileRows<1> - 1) / kTileRows<1>;
            tiles[1][i] = (n + kTileRows<2> - 1) / kTileRows<2>;
        }
        sum[0] += tiles[0][i];
        sum[1] += tiles[1][i];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        incl[h] = wave_inclusive_sum(sum[h]);
        if (lane == kWave - 1) t.wave_sum[h][wave] = incl[h];
    }
    __syncthreads();
    int run[2], total[2] = {0, 0};
    uint32_t most[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        run[h] = incl[h] - sum[h];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int s = t.wave_sum[h][w];
            if (w < wave) run[h] += s;
            total[h] += s;
        }
        total[h] = uniform(total[h]);
        most[h] = ((uint32_t)total[h] * n_tiles + gridDim.x - 1) / gridDim.x;
    }
    const int h = 7 * most[1] < 5 * most[0] ? 1 : 0;
    int r = h ? run[1] : run[0];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        r += h ? tiles[1][i] : tiles[0][i];
        if (e0 + i < p.E) t.end[e0 + i] = r;
    }
    __syncthreads();
    return Tiling{h ? total[1] : total[0], h + 1};
}

// The tiles of all experts in one row, an expert's tiles in groups of kGroup row tiles: within a
// group the row tile runs fastest, then the column tile. Neighbours in this order share weights
// and rows, and each XCD takes one eighth of the order (its workgroups are blockIdx.x mod 8), so
// that its L2 holds what they share. Groups of 4: 65536 rows x 4096 x 4096 1.17 ms; of 8 1.21 ms, of
// 16 1.25 ms (SwiGLU of the same rows: within 1%).
constexpr int kGroup = 4;

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

// Sixteen values as bf16 pairs, NaN as 0x7FC0 (the conversion instruction would keep its payload).
__device__ __forceinline__ void bf16_pairs(const f32x16 &v, uint32_t (&d)[8])
{
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) nan |= __builtin_isunordered(v[2 * i], v[2 * i + 1]);
    if (__any(nan)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = bf16_rne(v[2 * i]) | (bf16_rne(v[2 * i + 1]) << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
    }
}

// The SwiGLU epilogue of one tile of ROWS rows x 128 channels of h: the block amax meets in LDS, the
// codes go out through LDS in whole rows. A wavefront holds quarter `part` of the 128 channels, a
// lane G groups of 4 consecutive ones (group g at channel part * 32 + channel(g)) of M rows
// (row(m)), GROUP lanes apart from the other channels of the row.
template <int ROWS>
struct SwigluShared {
    uint32_t amax[4][ROWS];
    float scale[ROWS];
    u32x4 code[ROWS][8];
};

template <int ROWS, int M, int G, int GROUP, typename Row, typename Channel>
__device__ __forceinline__ void store_swiglu(SwigluShared<ROWS> &sh, float (&h)[M][G][4],
                                             int wave, int lane, int part, Row row,
                                             Channel channel,
                                             const ExpertProduct &p, int row0, int n, int nblk)
{
    const int thread = wave * kWave + lane;
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
        if (lane < GROUP) sh.amax[part][row(m)] = amax;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int r = row(m);
        uint32_t amax = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) amax = max(amax, sh.amax[w][r]);
        const float scale = block_scale(amax);
        // 2^-60 <= amax < inf: the quotients lie where div_by_rcp and the conversion are exact
        const bool plain = __any(amax < 0x21800000u || amax >= 0x7F800000u);
        const float y = 1.0f / scale;
        // chunk c of row r at place c ^ (r & 7): the lanes of a store are rows, 128 bytes apart
        auto put = [&](int g, uint32_t code) {
            const int w = part * 8 + (channel(g) >> 2);
            reinterpret_cast<uint32_t *>(&sh.code[r][(w >> 2) ^ (r & 7)])[w & 3] = code;
        };
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
                put(g, encode4_any(v, scale));
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g)
                put(g, e4m3_pack4(div_by_rcp(h[m][g][0], scale, y), div_by_rcp(h[m][g][1], scale, y),
                                  div_by_rcp(h[m][g][2], scale, y), div_by_rcp(h[m][g][3], scale, y)));
        }
        if (part == 0 && lane < GROUP) sh.scale[r] = scale;
    }
    __syncthreads();
    const int I = p.n / 2;
    for (int i = thread; i < ROWS * 8; i += kTileThreads) {
        const int r = i >> 3;
        if (r < n)
            *reinterpret_cast<u32x4 *>(p.h_q + (size_t)(row0 + r) * I + nblk * 128 + (i & 7) * 16) =
                sh.code[r][(i & 7) ^ (r & 7)];
    }
    for (int r = thread; r < n; r += kTileThreads)
        p.h_scale[(size_t)(row0 + r) * (I / 128) + nblk] = sh.scale[r];
    __syncthreads();
}

// Both kernels: tiles of 64 * MT rows x 256 weight rows (SwiGLU: 128 gate and the same 128 up rows),
// one workgroup of 8 wavefronts per CU that walks its tiles as one stream of blocks (128 channels of
// a tile each); a wavefront multiplies 32 * MT rows by 64 weight rows. Two wavefronts per SIMD share
// its issue slots: one alone issues an instruction in about 5 cycles, and its scaled sums and LDS
// reads then take longer than the products they should hide behind. Loads run ahead across tiles, so
// that neither a block nor a tile waits for memory. A load instruction covers 8 whole 128-byte row
// segments, 8 lanes a row: the vector cache takes one access per 128 bytes (in the matrix
// instruction's lane order, 16 rows side by side, it took one per 16 bytes, and that bounded every
// size: with operands straight from global memory to registers, 65536 rows x 4096 x 4096 took
// 4.7 ms, and 640 rows over 128 experts, 1536 x 2048, 84 us against 76 us). The row scales of some
// blocks are staged together, one panel ahead. One barrier per block.
//
// In LDS, chunk c (16 bytes) of row r is kept at place c ^ swizzle(r) of the row's eight: the lanes
// that LDS serves together (8 consecutive rows, and the same 16 further on) then touch all banks. A
// lane's j-th chunk of a block is 2 * j + half of row lane & 31.
__device__ __forceinline__ int swizzle(int r) { return (r & 7) ^ ((r >> 4) & 1); }

// The SwiGLU form. Its products, in bf16, keep the matrix units busier than the loads (65536 rows x
// 2 x 2048 x 4096: 2.05 ms, 83% of the rate of a large bf16 product on the same card), and the codes'
// conversion takes registers: loads go to registers, up to two blocks ahead, and from there to one of
// two LDS buffers, an eighth per wavefront.
constexpr int kPanel = 16;         // blocks whose scales are staged together
constexpr int kList = 256;         // tiles of a workgroup looked up together

// A buffer of `bytes` from p: loads take a lane offset and a uniform one, and give 0 past the end.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00027000);
}

__device__ __forceinline__ i32x4 buffer_load16(__amdgpu_buffer_rsrc_t b, int lane_off, int off)
{
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_off, off, 0));
}

// Meet the other wavefronts with LDS settled; loads in flight stay in flight.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The same with at most N of this wavefront's vector memory operations left (they finish in order).
template <int N>
__device__ __forceinline__ void meet_loaded()
{
    static_assert(N < 64, "the counter's range");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));    // vmcnt(N) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int MT>
struct SwigluTiles {
    static constexpr int kTileM = kTileRows<MT>;
    u32x4 x[2][kTileM * 8];
    u32x4 w[2][kTileN * 8];
    float xscale[2][kPanel][kTileM + 1];
    float wscale[2][kPanel][2];
    int4 list[kList];
    SwigluShared<kTileM> h;
};

template <int MT>
__device__ __forceinline__ void run_swiglu(const ExpertProduct &p, const TileTable &table,
                                           SwigluTiles<MT> &sh, int row_tiles)
{
    constexpr int kTileM = kTileRows<MT>;
    const int wave = uniform(threadIdx.x / kWave), lane = lane_now();
    const int wm = wave & 1, wn = wave >> 1;   // the wavefront's rows and weight rows
    const int r32 = lane & 31, half = lane >> 5;
    const int nkb = p.H >> 7;
    const int n_tiles = p.n / kTileN, ws_rows = p.n >> 7;
    const TileRange mine = my_tiles(row_tiles * n_tiles);
    const int row_at = r32 * 8, row_swizzle = swizzle(r32);

    // the stream of loads: the tile it is in and its next block
    struct {
        int tile, kb;
        __amdgpu_buffer_rsrc_t w, x;
        int woff[4], xoff[MT];
    } ld;
    // Weight row i of a tile: 32 gate rows and the same 32 up rows together, so that every wavefront
    // has a tile of each.
    auto weight_row = [&](int nblk, int i) {
        return ((i >> 5) & 1) * (p.n / 2) + nblk * 128 + (i >> 6) * 32 + (i & 31);
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
        const int l = lane_now();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ld.woff[j] = weight_row(t.nblk, wave * 32 + j * 8 + (l >> 3)) * p.H + (l & 7) * 16;
#pragma unroll
        for (int j = 0; j < MT; ++j)
            ld.xoff[j] = min(wave * (8 * MT) + j * 8 + (l >> 3), t.n - 1) * p.H + (l & 7) * 16;
    };

    // blocks in registers on their way to LDS, as many as there is room for (with one, 128 tokens over
    // 128 experts 82 us, with two 79)
    constexpr int kStage = MT == 2 ? 1 : 2;
    i32x4 wr[kStage][4], xr[kStage][MT];
    i32x4 wf[2][4];                            // the wavefront's weights of a block: [tile][chunk]
    f32x16 acc[2][MT];
    i32x4 xf[4];
    float xs[2];                               // row scales
    constexpr int kPer = kTileM * kPanel / kTileThreads;
    float ps[kPer], pw = 0.0f;                 // the next panel on its way
    int par = 0;                               // the panel in use

    auto load_w = [&](int d, int j) { wr[d % kStage][j] = buffer_load16(ld.w, ld.woff[j], ld.kb * 128); };
    auto load_x = [&](int d, int j) { xr[d % kStage][j] = buffer_load16(ld.x, ld.xoff[j], ld.kb * 128); };
    // the lane's place in LDS: its row of each 8, its chunk (rows 16 further on swap neighbours)
    auto place = [](int l) { return (l >> 3) * 8 + ((l & 7) ^ (l >> 3)); };
    const int put0 = place(lane);
    auto put_w = [&](int d, int j, int at) {
        sh.w[d][wave * 256 + j * 64 + (at ^ (j >> 1))] = __builtin_bit_cast(u32x4, wr[d % kStage][j]);
    };
    auto put_x = [&](int d, int j, int at) {
        sh.x[d][(wave * MT + j) * 64 + (at ^ ((wave * MT >> 1) & 1))] =
            __builtin_bit_cast(u32x4, xr[d % kStage][j]);
    };
    auto advance = [&](int tiles) {            // past the last block: that block again
        if (++ld.kb == nkb) {
            if (ld.tile + 1 < tiles) enter(ld.tile + 1);
            else ld.kb = nkb - 1;
        }
    };
    auto panel_load = [&](int i, int kb0) {
        const Tile t = at(i);
        const int l = wave * kWave + lane_now();
        const float *src = p.scale + (size_t)t.row0 * nkb + min(kb0 + (l & 15), nkb - 1);
#pragma unroll
        for (int k = 0; k < kPer; ++k) ps[k] = src[(size_t)min(k * 32 + (l >> 4), t.n - 1) * nkb];
        const int blk = ((l >> 4) & 1) * (p.n >> 8) + t.nblk;
        pw = (p.w_scale + (size_t)t.e * ws_rows * nkb)[blk * nkb + min(kb0 + (l & 15), nkb - 1)];
    };
    auto panel_store = [&](int to) {
        const int l = wave * kWave + lane_now();
#pragma unroll
        for (int k = 0; k < kPer; ++k) sh.xscale[to][l & 15][k * 32 + (l >> 4)] = ps[k];
        if (l < 32) sh.wscale[to][l & 15][l >> 4] = pw;
    };
    auto read_row = [&](int d, int mt) {       // the lane's chunks of row tile mt
        const i32x4 *x = reinterpret_cast<const i32x4 *>(sh.x[d]) + (wm * MT + mt) * 256 + row_at;
#pragma unroll
        for (int j = 0; j < 4; ++j) xf[j] = x[(2 * j + half) ^ row_swizzle];
    };
    auto read_w = [&](int d, int nt) {         // and of the wavefront's weight tile nt
        const i32x4 *w = reinterpret_cast<const i32x4 *>(sh.w[d]) + (wn * 2 + nt) * 256 + row_at;
#pragma unroll
        for (int j = 0; j < 4; ++j) wf[nt][j] = w[(2 * j + half) ^ row_swizzle];
    };
    float ws[2];                               // weight scales, gate and up
    auto read_ws = [&](float (&to)[2], int b) {
        to[0] = sh.wscale[par][b][0];
        to[1] = sh.wscale[par][b][1];
    };
    auto clear = [&]() {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[nt][mt][i] = 0.0f;
    };
    // One block, in LDS buffer d, in MT regions of one tile of 32 rows each, kept apart by fences. The
    // next block goes to LDS before the barrier, and the one kStage further takes its registers.
    auto step = [&](int d, int tile, int kb, int tiles) {
        const int dn = d ^ 1;
        if ((kb & (kPanel - 1)) == 0) {
            if (kb + kPanel < nkb) panel_load(tile, kb + kPanel);
            else if (tile + 1 < tiles) panel_load(tile + 1, 0);
        }
        const int b_next = kb == nkb - 1 ? 0 : (kb + 1) & (kPanel - 1);
        float ws_next[2];
        bf16x8 wb[2][8];
        read_w(d, 0);
        read_w(d, 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            read_row(d, mt);
            xs[mt] = sh.xscale[par][kb & (kPanel - 1)][(wm * MT + mt) * 32 + r32];
            if (mt == 0) {
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    put_x(dn, j, put0);
                    load_x(dn, j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    put_w(dn, j, put0);
                    load_w(dn, j);
                }
            }
            if (mt == MT - 1) {
                if (b_next == 0) {
                    par ^= 1;
                    panel_store(par);
                }
                meet();
                read_ws(ws_next, b_next);
            }
            f32x16 v[2] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bf16x8 xb = bf16_of_e4m3(xf[j >> 1][(j & 1) * 2], xf[j >> 1][(j & 1) * 2 + 1]);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    if (mt == 0)
                        wb[nt][j] = bf16_of_e4m3(wf[nt][j >> 1][(j & 1) * 2],
                                                 wf[nt][j >> 1][(j & 1) * 2 + 1]);
                    v[nt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[nt][j], xb, v[nt], 0, 0, 0);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const float s = xs[mt] * ws[nt];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[nt][mt][i] = __builtin_fmaf(s, v[nt][i], acc[nt][mt][i]);
                asm volatile("" : "+v"(acc[nt][mt]));    // summed here, not later
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) ws[i] = ws_next[i];
        advance(tiles);
    };
    auto finish = [&](int tile) {              // the tile's output
        const Tile t = at(tile);
        const int l = lane_now();
        // element i of a lane is channel (i >> 2) * 8 + half * 4 + (i & 3) of row lane & 31
        float h[MT][4][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 16; ++i) h[mt][i >> 2][i & 3] = swiglu(acc[0][mt][i], acc[1][mt][i]);
        store_swiglu<kTileM, MT, 4, 32>(
            sh.h, h, wave, l, wn, [&](int m) { return (wm * MT + m) * 32 + (l & 31); },
            [&](int g) { return g * 8 + (l >> 5) * 4; }, p, t.row0, t.n, t.nblk);
        clear();
    };

#pragma unroll
    for (int k = 0; k < kPer; ++k) ps[k] = 0.0f;
    for (int first = mine.first; first < mine.end; first += kList * mine.step) {
        const int tiles = min((mine.end - first + mine.step - 1) / mine.step, kList);
        if (const int i = wave * kWave + lane_now(); i < tiles) {
            int columns;                       // nothing of its divisions stays in registers
            asm volatile("" : "=s"(columns) : "0"(uniform(n_tiles)));
            const Tile t = locate(table, p.E, first + i * mine.step, columns, kTileM);
            sh.list[i] = int4{t.e, t.row0, t.n, t.nblk};
        }
        __syncthreads();
        enter(0);
        par = 0;
        panel_load(0, 0);
        auto load = [&](int d) {
#pragma unroll
            for (int j = 0; j < MT; ++j) load_x(d, j);
#pragma unroll
            for (int j = 0; j < 4; ++j) load_w(d, j);
            advance(tiles);
        };
        load(0);
        if constexpr (kStage == 2) load(1);
        panel_store(0);
        const int put1 = place(lane_now());
#pragma unroll
        for (int j = 0; j < MT; ++j) put_x(0, j, put1);
#pragma unroll
        for (int j = 0; j < 4; ++j) put_w(0, j, put1);
        load(0);
        meet();
        read_ws(ws, 0);
        clear();
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
}

// The bf16 product. A block's rows and weights go from global memory to LDS directly, into one of three
// stages, and take no registers on the way: they hold instead three products on their way to the
// sums, so that the sums of a product run beside the two after it, and the next block's weights and
// rows, read behind the products that used this block's. The three stages are variables of their own:
// by that the compiler can tell a stage's reads from the loads in flight into another, and does not
// wait for those. The loads of the block three ahead start at the barrier behind which no wavefront
// reads the stage any more, a few at a time: all at once they held up the issue of everything else
// (65536 rows x 4096 x 4096: 1.34 ms; spread over a block's products 1.26 ms; with 8 wavefronts rather
// than 4 of 64 * MT rows x 128 weight rows 1.23 ms; with what tiles' order and stores gain 1.15 ms,
// 62% of the rate of a large FP8 product. At 1.23 ms the loads cost 0.24 ms, mostly of waiting for what
// misses L2, and the reads of LDS 0.1 ms).
constexpr int kGemmPanel = 8;      // blocks whose scales are staged together

typedef __attribute__((address_space(3))) uint8_t *LdsBytes;

struct GemmShared {
    float xscale[2][kGemmPanel][kTileRows<2> + 1];
    float wscale[2][kGemmPanel][2];
    int4 list[kList];
};

template <int MT, typename Stage>
__device__ __forceinline__ void run_gemm(const ExpertProduct &p, const Stage &stage, GemmShared &sh,
                                         int tiles)
{
    constexpr int kRows = kTileRows<MT>;
    constexpr int kW = kRows * 128;            // a stage: rows, then weights
    const int wave = uniform(threadIdx.x / kWave), lane = lane_now();
    const int wm = wave & 1, wn = wave >> 1;
    const int r32 = lane & 31, half = lane >> 5;
    const int nkb = p.H >> 7;
    const int ws_rows = (p.n + 127) >> 7;
    const int row_at = r32 * 8, row_swizzle = swizzle(r32);

    struct {
        int tile, kb;
        __amdgpu_buffer_rsrc_t w, x;
        int woff[4], xoff[MT];
    } ld;
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
        // a direct load fills 8 rows, lane l place l & 7 of row l >> 3: it loads the chunk kept there
        const int l = lane_now();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ld.woff[j] = min(t.nblk * kTileN + wave * 32 + j * 8 + (l >> 3), p.n - 1) * p.H +
                         ((l & 7) ^ (l >> 3) ^ (j >> 1)) * 16;
#pragma unroll
        for (int j = 0; j < MT; ++j)
            ld.xoff[j] = min(wave * 8 * MT + j * 8 + (l >> 3), t.n - 1) * p.H +
                         ((l & 7) ^ (l >> 3) ^ (((wave * MT + j) >> 1) & 1)) * 16;
    };
    constexpr int kLoads = 4 + MT;             // direct loads of a wavefront per block
    auto load_some = [&](uint8_t *to, int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            if (i < 4)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    ld.w, (LdsBytes)(to + kW + (wave * 4 + i) * 1024), 16, ld.woff[i], ld.kb * 128, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    ld.x, (LdsBytes)(to + (wave * MT + i - 4) * 1024), 16, ld.xoff[i - 4],
                    ld.kb * 128, 0, 0);
        }
    };
    auto advance = [&]() {                     // past the last block: that block again
        if (++ld.kb == nkb) {
            if (ld.tile + 1 < tiles) enter(ld.tile + 1);
            else ld.kb = nkb - 1;
        }
    };

    constexpr int kNT = 2, kQ = kNT * MT;      // tiles of 32 weight rows, products of a block
    f32x16 acc[kNT][MT];
    f32x16 v[3];                               // products on their way to acc
    i32x4 wf[kNT][4], xf[2][4];
    float sw[2], ws, xs[2];
    constexpr int kPer = kRows * kGemmPanel / kTileThreads;
    float ps[kPer], pw = 0.0f;                 // the next panel on its way
    int par = 0;                               // the panel in use
    auto panel_load = [&](int i, int kb0) {
        const Tile t = at(i);
        const int l = wave * kWave + lane_now();
        const float *src = p.scale + (size_t)t.row0 * nkb + min(kb0 + (l & 7), nkb - 1);
#pragma unroll
        for (int k = 0; k < kPer; ++k) ps[k] = src[(size_t)min(k * 64 + (l >> 3), t.n - 1) * nkb];
        const int blk = min(t.nblk * 2 + ((l >> 3) & 1), ws_rows - 1);
        pw = (p.w_scale + (size_t)t.e * ws_rows * nkb)[blk * nkb + min(kb0 + (l & 7), nkb - 1)];
    };
    auto panel_store = [&](int to) {
        const int l = wave * kWave + lane_now();
#pragma unroll
        for (int k = 0; k < kPer; ++k) sh.xscale[to][l & 7][k * 64 + (l >> 3)] = ps[k];
        if (l < 16) sh.wscale[to][l & 7][l >> 3] = pw;
    };
    auto read_row = [&](i32x4 (&to)[4], const uint8_t *from, int mt) {
        const i32x4 *x = reinterpret_cast<const i32x4 *>(from) + (wm * MT + mt) * 256 + row_at;
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = x[(2 * j + half) ^ row_swizzle];
    };
    auto read_w = [&](i32x4 (&to)[4], const uint8_t *from, int nt) {
        const i32x4 *w = reinterpret_cast<const i32x4 *>(from + kW) + (wn * kNT + nt) * 256 + row_at;
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = w[(2 * j + half) ^ row_swizzle];
    };
    auto read_xs = [&](int b, int mt) { return sh.xscale[par][b][(wm * MT + mt) * 32 + r32]; };
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[nt][mt][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < 3; ++k) v[k][i] = 0.0f;
        }
        sw[0] = sw[1] = 0.0f;
    };
    // sums half of product number q of a block (those before 0: the last ones of the block before)
    auto sum = [&](auto at_q, int ring, int parity, int h) {
        constexpr int q = (decltype(at_q)::value + 2 * kQ) % kQ;
        constexpr int nt = q % kNT, mt = q / kNT;
        const float f = sw[MT == 1 ? parity : mt];
#pragma unroll
        for (int i = h * 8; i < h * 8 + 8; ++i)
            acc[nt][mt][i] = __builtin_fmaf(f, v[ring][i], acc[nt][mt][i]);
        asm volatile("" : "+v"(acc[nt][mt]));            // summed here, not later
    };
    auto step = [&](auto at_s, auto at_p, int tile, int kb) {
        constexpr int S = decltype(at_s)::value, P = decltype(at_p)::value;
        constexpr int R = S * kQ % 3;         // ring place of the block's first product
        uint8_t *cur = stage(std::integral_constant<int, S>{});
        uint8_t *prev = stage(std::integral_constant<int, (S + 2) % 3>{});
        const uint8_t *nxt = stage(std::integral_constant<int, (S + 1) % 3>{});
        if ((kb & (kGemmPanel - 1)) == 0) {
            if (kb + kGemmPanel < nkb) panel_load(tile, kb + kGemmPanel);
            else if (tile + 1 < tiles) panel_load(tile + 1, 0);
        }
        const int b = kb & (kGemmPanel - 1), b_next = kb == nkb - 1 ? 0 : (kb + 1) & (kGemmPanel - 1);
        auto part = [&](auto at_q) {
            constexpr int q = decltype(at_q)::value, nt = q % kNT, mt = q / kNT;
            constexpr int X = MT == 1 ? P : mt;
            constexpr bool last = mt == MT - 1;
            if constexpr (last && nt == 0) {
                if (b_next == 0) {
                    par ^= 1;
                    panel_store(par);
                }
                // the next block's loads are done; those of the one after may be in flight
                meet_loaded<kLoads>();
            }
            f32x16 &to = v[(R + q) % 3];
            const f32x16 zero = {};
            const i32x8 x0 = join(xf[X][0], xf[X][1]), x1 = join(xf[X][2], xf[X][3]);
            to = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(wf[nt][0], wf[nt][1]), x0, zero, 0,
                                                                 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            sum(std::integral_constant<int, q - 2>{}, (R + q + 1) % 3, q < 2 ? P ^ 1 : P, 0);
            if constexpr (nt == 0 && !last) {
                read_row(xf[(mt + 1) & 1], cur, mt + 1);
                xs[(mt + 1) & 1] = read_xs(b, mt + 1);
            }
            // the loads of the block three ahead, from the barrier on for as many products as a
            // block has: MT = 2 ends them in the next block
            constexpr int since = (q + kNT) % kQ;               // products since the barrier
            constexpr int i0 = since * kLoads / kQ, i1 = (since + 1) * kLoads / kQ;
            load_some(last ? cur : prev, i0, i1);
            if constexpr (i1 == kLoads) advance();
            __builtin_amdgcn_sched_barrier(0);
            to = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(wf[nt][2], wf[nt][3]), x1, to, 0,
                                                                 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            sum(std::integral_constant<int, q - 2>{}, (R + q + 1) % 3, q < 2 ? P ^ 1 : P, 1);
            if constexpr (nt == 1) sw[X] = xs[X] * ws;     // the sums before it are done
            if constexpr (last) {
                if constexpr (nt == 0) {
                    read_row(xf[MT == 1 ? P ^ 1 : 0], nxt, 0);
                    xs[MT == 1 ? P ^ 1 : 0] = read_xs(b_next, 0);
                }
                read_w(wf[nt], nxt, nt);
                if constexpr (nt == kNT - 1) ws = sh.wscale[par][b_next][wn >> 1];
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        part(std::integral_constant<int, 0>{});
        part(std::integral_constant<int, 1>{});
        if constexpr (MT == 2) {
            part(std::integral_constant<int, 2>{});
            part(std::integral_constant<int, 3>{});
        }
    };
    auto finish = [&](auto at_s, auto at_p, int tile) {
        constexpr int R = decltype(at_s)::value * kQ % 3, P = decltype(at_p)::value;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum(std::integral_constant<int, -2>{}, (R + kQ - 2) % 3, P, h);
            sum(std::integral_constant<int, -1>{}, (R + kQ - 1) % 3, P, h);
        }
        const Tile t = at(tile);
        const int l = lane_now();
        // element i of a lane is channel (i >> 2) * 8 + half * 4 + (i & 3) of row lane & 31; the lanes'
        // halves trade, so that one stores the eight channels of an even i >> 2 and one those of the
        // odd one behind it (n % 8 == 0: all or none are there): 16 bytes a store instead of 8, 97 us
        // against 112 with 32768 rows x 768 x 2048, where an output comes every six blocks
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = (wm * MT + mt) * 32 + (l & 31), c0 = t.nblk * kTileN + wn * 64 + (l >> 5) * 8;
            uint16_t *y = p.y + (size_t)(t.row0 + r) * p.n + c0;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                uint32_t d[8];
                bf16_pairs(acc[nt][mt], d);
#pragma unroll
                for (int g = 0; g < 4; g += 2) {
                    const auto a = __builtin_amdgcn_permlane32_swap(d[2 * g], d[2 * g + 2], false, false);
                    const auto b = __builtin_amdgcn_permlane32_swap(d[2 * g + 1], d[2 * g + 3], false, false);
                    if (r < t.n && c0 + nt * 32 + g * 8 < p.n)
                        *reinterpret_cast<u32x4 *>(y + nt * 32 + g * 8) = u32x4{a[0], b[0], a[1], b[1]};
                }
            }
        }
        clear();
    };

#pragma unroll
    for (int k = 0; k < kPer; ++k) ps[k] = 0.0f;
    enter(0);
    panel_load(0, 0);
    panel_store(0);
    load_some(stage(std::integral_constant<int, 0>{}), 0, kLoads);
    advance();
    load_some(stage(std::integral_constant<int, 1>{}), 0, kLoads);
    advance();
    load_some(stage(std::integral_constant<int, 2>{}), 0, kLoads / MT);
    if constexpr (MT == 1) advance();
    constexpr int kAfter = kLoads + kLoads / MT;         // than the first block's
    meet_loaded<kAfter>();
    const uint8_t *first = stage(std::integral_constant<int, 0>{});
    read_row(xf[0], first, 0);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) read_w(wf[nt], first, nt);
    xs[0] = read_xs(0, 0);
    ws = sh.wscale[0][0][wn >> 1];
    clear();
    int tile = 0, kb = 0;
    auto next = [&](auto at_s, auto at_p) {    // a block; false after the last one
        step(at_s, at_p, tile, kb);
        if (++kb < nkb) return true;
        finish(at_s, at_p, tile);
        kb = 0;
        return ++tile < tiles;
    };
    std::integral_constant<int, 0> c0;
    std::integral_constant<int, 1> c1;
    std::integral_constant<int, 2> c2;
    while (next(c0, c0) && next(c1, c1) && next(c2, c0) && next(c0, c1) && next(c1, c0) && next(c2, c1)) {}
    meet_loaded<0>();                          // no direct load is left to write LDS
}
#endif

__global__ __launch_bounds__(kTileThreads) void expert_gemm_kernel(ExpertProduct p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(16))) uint8_t s0[(kTileRows<2> + kTileN) * 128];
    __shared__ __attribute__((aligned(16))) uint8_t s1[(kTileRows<2> + kTileN) * 128];
    __shared__ __attribute__((aligned(16))) uint8_t s2[(kTileRows<2> + kTileN) * 128];
    __shared__ GemmShared sh;
    static_assert(sizeof(TileTable) <= sizeof(s0), "the table is done with before the first block");
    auto stage = [&](auto s) -> uint8_t * {
        if constexpr (decltype(s)::value == 0) return s0;
        else if constexpr (decltype(s)::value == 1) return s1;
        else return s2;
    };
    TileTable &table = *reinterpret_cast<TileTable *>(s0);
    const int wave = uniform(threadIdx.x / kWave);
    const int n_tiles = (p.n + kTileN - 1) / kTileN;
    for (int done = 0;;) {                     // kList tiles at a time
        const Tiling t = build_table(table, p, n_tiles);
        const TileRange mine = my_tiles(t.total * n_tiles);
        const int first = mine.first + done * mine.step;
        if (first >= mine.end) break;
        const int tiles = min((mine.end - first + mine.step - 1) / mine.step, kList);
        if (const int i = wave * kWave + lane_now(); i < tiles) {
            int columns;                       // nothing of its divisions stays in registers
            asm volatile("" : "=s"(columns) : "0"(uniform(n_tiles)));
            const Tile l = locate(table, p.E, first + i * mine.step, columns, t.mt * 64);
            sh.list[i] = int4{l.e, l.row0, l.n, l.nblk};
        }
        __syncthreads();                       // the table is done with
        if (t.mt == 1) run_gemm<1>(p, stage, sh, tiles);
        else run_gemm<2>(p, stage, sh, tiles);
        done += tiles;
    }
#else
    (void)p;
#endif
}

__global__ __launch_bounds__(kTileThreads) void expert_swiglu_kernel(ExpertProduct p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ TileTable table;
    __shared__ union {
        SwigluTiles<1> low;
        SwigluTiles<2> high;
    } sh;
    const Tiling t = build_table(table, p, p.n / kTileN);
    if (t.mt == 1) run_swiglu<1>(p, table, sh.low, t.total);
    else run_swiglu<2>(p, table, sh.high, t.total);
#else
    (void)p;
#endif
}

constexpr int kCus = 256;

// One workgroup per CU, or as many as there can be tiles of 64 rows.
hipError_t launch_product(void (*kernel)(ExpertProduct), const ExpertProduct &p, hipStream_t stream)
{
    if (p.pairs == 0 || (p.offset && p.rows == 0)) return hipSuccess;
    const int64_t experts = p.pairs < p.E ? p.pairs : p.E;
    const int64_t tiles = (p.pairs / kTileRows<1> + experts) * ((p.n + kTileN - 1) / kTileN);
    const dim3 grid((unsigned)(tiles < kCus ? (tiles + 7) / 8 * 8 : kCus));
    return launch(kernel, grid, dim3(kTileThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_expert_gemm_fp8(const ExpertProduct &p, hipStream_t stream)
{
    return launch_product(expert_gemm_kernel, p, stream);
}

hipError_t launch_expert_swiglu_fp8(const ExpertProduct &p, hipStream_t stream)
{
    return launch_product(expert_swiglu_kernel, p, stream);
}

}  // namespace ep
