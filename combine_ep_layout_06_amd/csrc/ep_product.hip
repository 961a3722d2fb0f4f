// The bf16 products on gfx950: the experts' product and its two gradients, the same with SwiGLU or its
// gradient in the epilogue, and the dense product with bias, activation and residual.
//
//   forward   out[r][c]    = sum_k x[r][k] w[e][c][k]
//   dgrad     out[r][c]    = sum_k x[r][k] w[e][k][c]
//   wgrad     out[e][r][c] = sum_i x[i][r] w[i][c]       i over the rows of expert e
//
// One kernel for the three. A tile is 256 rows x 256 columns of the output, in blocks of 64 of the sum:
// a workgroup of 8 wavefronts per CU walks its tiles as one stream of blocks, loads running ahead
// across tiles, each wavefront with 128 x 64 of the tile in 128 registers (32 x 32 x 16 matrix
// instructions; w is the A operand, so that a lane holds one row and groups of four columns). Of a
// tile with fewer rows the wavefronts multiply only the parts of 64 that hold some.
//
// Operands go from global memory to LDS directly, in two stages of a block each, and a block in halves
// of 128 rows or columns. An operand whose sum index runs along its rows in memory is kept row by row,
// 128 bytes of a row, and read 16 bytes a lane. One whose sum index is the row number is kept as it
// lies, 64 rows of 128 values, and read with the transposing LDS read, which gives a lane four
// consecutive sum indexes of one column.
//
// A block is four phases of a quarter of its products. In each a wavefront reads from LDS what the next
// phase needs and starts loading one of the four halves of the block after the next into the place of
// one that all have read: so the loads are spread evenly, and every one has six phases to arrive.
//
// 65536 rows x 4096 x 4096: a meeting of the wavefronts a block 1.86 ms, four phases 1.79, outputs stored
// 64 bytes of a row together, which no later load waits for, 1.66, one stream of loads through tiles of
// different heights 1.62 (1.36 PFLOP/s; matrix units 77% busy at the 1.6-1.75 GHz that the load leaves).
// With short sums and some 340 rows an expert (two row tiles of 192) a round of tiles is its blocks and then
// its output, beside which nothing runs. 96 experts of 2048 columns, sums of 256 to 4096 (kernel times): a
// block 1.4-1.55 us (10 TB/s into LDS, 1.1 PFLOP/s, 3.3 TB/s from HBM if all is read once), the output of
// a round 4 us, with gu 7, SwiGLU's gradient 22 (100 MB of gu and dgu: a copy's rate). Of experts
// with one row tile a block takes 1.6-2.4, the weights' read (4.4 TB/s of 64 rows); of one matrix that the
// caches hold 0.65 for 64 rows (16 TB/s into LDS, which is not what bounds the others). Cutting a last
// round's tiles and groups of about 8 row tiles took 4096 tokens' gate and up products from 275 to 259 us and
// their down gradients from 308 to 286.
// Blocks of 32 in four stages (64 bytes of a row, twice the L2 requests), other cache policies of loads or
// stores (0-15% slower), groups of 4 or 16, a raised wave priority: slower or no gain.
#include "ep_product.h"

#include <type_traits>

namespace ep {

namespace {

constexpr int kThreads = 512;
constexpr int kTile = 256;         // rows and columns of a tile
constexpr int kPart = 64;          // rows of a part
constexpr int kCus = 256;

namespace form { constexpr int kForward = 0, kDgrad = 1, kWgrad = 2; }
namespace to { constexpr int kBf16 = 0, kSwiglu = 1, kSwigluGrad = 2, kF32 = 3, kLinear = 4; }

#if defined(__HIP_DEVICE_COMPILE__)            // buffer descriptors exist on the device only

constexpr int kWaves = kThreads / kWave;
constexpr int kBlock = 64;         // sum indexes of a block
constexpr int kHalf = kTile / 2 * kBlock * 2;    // bytes of half an operand of a block
constexpr int kStage = 4 * kHalf;  // of a block: x's halves, w's halves
constexpr int kLoads = 8;          // of a block, by one wavefront
constexpr int kList = kWave;       // tiles of a workgroup looked up together

using ep::uniform;

// The experts' rows cut into row tiles: rows and first row of each expert and the running number of row
// tiles.
struct TileTable {
    int32_t end[EP_MAX_EXPERTS], base[EP_MAX_EXPERTS], n[EP_MAX_EXPERTS];
    int32_t wave_sum[kWaves];
};

__device__ __forceinline__ void rows_of(const Product &p, int e, int &base, int &n)
{
    if (!p.count || p.pairs == 0) {            // dense, or no rows: the arrays need not be there
        base = 0;
        n = p.pairs == 0 ? 0 : p.C;
    } else {
        expert_rows(p.count, p.offset, e, p.C, p.rows, base, n);
    }
}

__device__ __forceinline__ int tiles_of(int n) { return ((uint32_t)n + kTile - 1) / kTile; }

// First part of tile i of an expert with n rows: its parts spread evenly over its tiles, the larger ones
// first.
__device__ __forceinline__ int first_part(int n, int i)
{
    const int parts = ((uint32_t)n + kPart - 1) / kPart, tiles = max(tiles_of(n), 1), each = parts / tiles;
    return i * each + min(i, parts - tiles * each);
}

__device__ __forceinline__ int build_table(TileTable &t, const Product &p)
{
    constexpr int kPer = EP_MAX_EXPERTS / kThreads;
    const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
    const int e0 = threadIdx.x * kPer;
    int tiles[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        tiles[i] = 0;
        if (e0 + i < p.E) {
            int base, n;
            rows_of(p, e0 + i, base, n);
            t.base[e0 + i] = base;
            t.n[e0 + i] = n;
            tiles[i] = tiles_of(n);
        }
        sum += tiles[i];
    }
    const int incl = wave_inclusive_sum(sum);
    if (lane == kWave - 1) t.wave_sum[wave] = incl;
    __syncthreads();
    int run = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
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
    return uniform(total);
}

// A tile: columns from nblk * kTile of the output, `rows` rows (0: no tile). Forward and dgrad: rows row0
// .. row0 + n of expert e, n = rows. Wgrad: rows m0 .. of expert e's output, and the sum is over the
// rows row0 .. row0 + n.
struct Tile {
    int e, row0, n, nblk, m0, rows;
};

// The tile at place `at` of the order: an expert's tiles in groups of about 8 row tiles, within a group
// the row tile runs fastest, then the column tile. Tiles side by side in this order share operands.
__device__ __forceinline__ Tile locate(const TileTable &t, const Product &p, int at, int n_tiles)
{
    const int m = at / n_tiles;
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.end[mid] > m) hi = mid;
        else lo = mid + 1;
    }
    const int n_e = t.n[lo], tiles = tiles_of(n_e);
    const int groups = max((tiles + 4) / 8, 1), size = (tiles + groups - 1) / groups;
    at -= (t.end[lo] - tiles) * n_tiles;
    const int group = at / (size * n_tiles), in_group = min(tiles - group * size, size);
    at -= group * size * n_tiles;
    Tile r;
    r.e = lo;
    r.nblk = at / in_group;
    const int m_tile = group * size + at - r.nblk * in_group;
    const int first = first_part(n_e, m_tile) * kPart;
    r.row0 = t.base[lo] + first;
    r.n = r.rows = min((uint32_t)first_part(n_e, m_tile + 1) * kPart, (uint32_t)n_e) - first;
    r.m0 = 0;
    return r;
}

__device__ __forceinline__ Tile locate_wgrad(const Product &p, int at, int m_tiles, int n_tiles)
{
    Tile r;
    r.e = at / (m_tiles * n_tiles);
    at -= r.e * m_tiles * n_tiles;
    r.nblk = at / m_tiles;
    const int m_tile = at - r.nblk * m_tiles;
    r.m0 = first_part(p.m, m_tile) * kPart;
    r.rows = min(first_part(p.m, m_tile + 1) * kPart, p.m) - r.m0;
    rows_of(p, r.e, r.row0, r.n);
    return r;
}

// One of `cuts` pieces of a tile, whole parts of its rows.
__device__ __forceinline__ void cut(Tile &t, int piece, int cuts, bool wgrad)
{
    const int parts = (t.rows + kPart - 1) / kPart;
    const int first = piece * parts / cuts * kPart;
    t.rows = min((piece + 1) * parts / cuts * kPart, t.rows) - first;
    if (wgrad) {
        t.m0 += first;
    } else {
        t.row0 += first;
        t.n = t.rows;
    }
}

// Meet the other wavefronts with this one's LDS reads done, and all but its last N loads.
template <int N>
__device__ __forceinline__ void meet_loaded()
{
    static_assert(N < 64, "the counter's range");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));    // vmcnt(N) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Two values as bf16, rounded to nearest even (a NaN stays one).
__device__ __forceinline__ uint32_t pair(float a, float b)
{
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

__device__ __forceinline__ u32x4 pack8(const float (&v)[8])
{
    return u32x4{pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])};
}

// Rows of an output (or of an epilogue's input) of a tile: `n` rows of `ld` values of `size` bytes. Lanes
// address them by byte offsets; those of rows that are not there, and kNone, lie past the end, where
// nothing is stored and loads give 0.
struct Rows {
    __amdgpu_buffer_rsrc_t b;
    __device__ __forceinline__ Rows(const void *p, size_t row0, int n, int ld, int size)
    {
        const uint8_t *at = reinterpret_cast<const uint8_t *>(p) + row0 * ld * size;
        b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(at), 0, n * ld * size, 0x00027000);
    }
    __device__ __forceinline__ void put(uint32_t off, u32x4 v) const
    {
        __builtin_amdgcn_raw_buffer_store_b128(v, b, off, 0, 0);
    }
    __device__ __forceinline__ u32x4 get(uint32_t off) const
    {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
    }
};

// Swizzle of row r of an operand kept row by row: chunk c (16 bytes) of the row's eight is at place
// c ^ swizzle(r). LDS serves 16 lanes together, 8 consecutive rows and those 16 further on: they then
// touch all banks once.
__device__ __forceinline__ int swizzle(int r) { return (r & 7) ^ ((r >> 4) & 1); }

// In one kept as it lies the 64-byte unit u of row k's four is at place u ^ (k & 3): the four rows whose
// units a transposing read of 32 lanes takes then lie in different banks.

// The stream of loads of a workgroup's tiles, kept up from tile to tile: the tile it is in and its next
// block, and the stage that the products are in.
template <int F, int O>
struct Stream {
    static constexpr bool kXTr = F == form::kWgrad, kWTr = F != form::kForward;
    const Product &p;
    const Tile *list;
    int tiles;
    uint32_t stage = 0;                        // byte offset
    int stored = 0;                            // barriers to come whose loads are older than stores
    int parts = 0;                             // of the tile that made these
    int tile, kb, nkb;
    const uint8_t *x, *w;
    int64_t xleft, wleft;                      // bytes from x and w to the operands' ends
    i32x4 xb, wb;
    uint32_t xoff, woff;
    uint64_t beyond;                           // lanes whose chunk of a row's last block is beyond the row

    __device__ __forceinline__ int wave() const { return uniform(threadIdx.x / kWave); }
    __device__ __forceinline__ int ldx() const { return F == form::kWgrad ? p.m : p.k; }
    __device__ __forceinline__ int ldw() const { return F == form::kForward ? p.k : p.n; }
    // A load of an operand kept row by row fills 8 rows of 8 chunks, one of an operand kept as it lies 4
    // rows of 16; a wavefront makes two of each half.
    __device__ __forceinline__ int chunk_of(int l) const { return (l & 7) ^ (l >> 3) ^ (wave() & 1); }

    __device__ __forceinline__ Stream(const Product &p, const Tile *list, int tiles)
        : p(p), list(list), tiles(tiles)
    {
        const int tail = (p.k & (kBlock - 1)) ? (p.k & (kBlock - 1)) / 8 : 8;
        beyond = __ballot(chunk_of(lane_now()) >= tail);
        enter(0);
    }
    __device__ __forceinline__ Tile at(int i) const
    {
        const Tile t = list[i];
        return Tile{uniform(t.e), uniform(t.row0), uniform(t.n), uniform(t.nblk), uniform(t.m0), uniform(t.rows)};
    }
    __device__ __forceinline__ int blocks_of(const Tile &t) const
    {
        return F == form::kWgrad ? max((int)(((uint32_t)t.n + kBlock - 1) / kBlock), 1) : (p.k + kBlock - 1) / kBlock;
    }
    __device__ __forceinline__ void enter(int i)
    {
        const Tile t = at(i);
        tile = i;
        kb = 0;
        nkb = blocks_of(t);
        if constexpr (F == form::kForward) {
            w = reinterpret_cast<const uint8_t *>(p.w + (size_t)t.e * p.n * p.k);
            wleft = (int64_t)p.n * p.k * 2;
        } else if constexpr (F == form::kDgrad) {
            w = reinterpret_cast<const uint8_t *>(p.w + (size_t)t.e * p.n * p.k + t.nblk * kTile);
            wleft = ((int64_t)p.n * p.k - t.nblk * kTile) * 2;
        } else {
            w = reinterpret_cast<const uint8_t *>(p.w + (size_t)t.row0 * p.n + t.nblk * kTile);
            wleft = ((int64_t)t.n * p.n - t.nblk * kTile) * 2;
        }
        x = reinterpret_cast<const uint8_t *>(p.x + (size_t)t.row0 * ldx() + t.m0);
        xleft = ((int64_t)t.n * ldx() - t.m0) * 2;
        xb = buffer(x, xleft);
        wb = buffer(w, wleft);
        const int l = lane_now(), chunk = chunk_of(l);
        const int row8 = wave() * 16 + (l >> 3), row4 = wave() * 8 + (l >> 4);
        const int tr_byte = ((((l >> 2) ^ (l >> 4)) & 3) << 6) + (l & 3) * 16;
        const int wrow = t.nblk * (O == to::kSwiglu ? kTile / 2 : kTile) + row8;
        if constexpr (kXTr) xoff = (uint32_t)row4 * ldx() * 2 + tr_byte;
        else xoff = (uint32_t)row8 * ldx() * 2 + chunk * 16;
        if constexpr (kWTr) woff = (uint32_t)row4 * ldw() * 2 + tr_byte;
        else woff = (uint32_t)wrow * ldw() * 2 + chunk * 16;
    }
    // One half of an operand of the block to the stage at byte offset `to`: past an operand's end the
    // loads give 0.
    template <bool W>
    __device__ __forceinline__ void load(uint8_t *stages, uint32_t to, int half_no)
    {
        constexpr bool TR = W ? kWTr : kXTr;
        uint8_t *at = stages + to + (2 * W + half_no) * kHalf + wave() * 2048;
        const int ldm = W ? ldw() : ldx();
        uint32_t off = W ? woff : xoff;
        if (!TR && __builtin_amdgcn_inverse_ballot_w64(kb == nkb - 1 ? beyond : 0)) off = kNone;
        uint32_t soff = TR ? half_no * 256 : kb * (kBlock * 2);
        if (!TR && half_no)                    // SwiGLU: the second half are the up rows
            soff += (W && O == to::kSwiglu ? (uint32_t)(p.n / 2) : 128u) * ldm * 2;
        load_lds(W ? wb : xb, at, off, soff);
        load_lds(W ? wb : xb, at + 1024, off, soff + (TR ? 8 : 16) * ldm);
    }
    __device__ __forceinline__ void advance()  // past the last block: that block again
    {
        if (kb + 1 < nkb) {
            ++kb;
            if constexpr (kXTr) {
                x += (size_t)kBlock * ldx() * 2;
                xleft -= (int64_t)kBlock * ldx() * 2;
                xb = buffer(x, xleft);
            }
            if constexpr (kWTr) {
                w += (size_t)kBlock * ldw() * 2;
                wleft -= (int64_t)kBlock * ldw() * 2;
                wb = buffer(w, wleft);
            }
        } else if (tile + 1 < tiles) {
            enter(tile + 1);
        }
    }
    // The first two blocks; the first one's first halves are there when it returns.
    __device__ __forceinline__ void start(uint8_t *stages)
    {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            load<false>(stages, b * kStage, 0);
            load<true>(stages, b * kStage, 0);
            load<true>(stages, b * kStage, 1);
            load<false>(stages, b * kStage, 1);
            advance();
        }
        meet_loaded<2 * kLoads - 4>();
    }
};

// Tiles `tile` .. `end` of the stream, which all have A parts.
template <int F, int O, int A>
__device__ __forceinline__ void run(Stream<F, O> &ld, uint8_t *stages, int tile, int end)
{
    constexpr bool kXTr = F == form::kWgrad, kWTr = F != form::kForward;
    const int wave = ld.wave(), wm = wave & 1, wn = wave >> 1;

    f32x16 acc[2][A];
    bf16x8 wf[2][4], xf[A][4];                 // 16 sum indexes each
    auto clear = [&]() {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int mt = 0; mt < A; ++mt)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[nt][mt][i] = 0.0f;
    };
    // Where a lane reads sum indexes 0 .. of its wavefront's first 32 rows (columns) in a half. Row by row:
    // chunk 2 * j + half of row lane & 31 for those from 16 * j on. As it lies: rows half * 8 + 0 .. 3
    // (and, 4 rows further, the rest), its 16 lanes' part of a unit. One address for each j, or for each
    // of x's two units, that steps from stage to stage.
    constexpr int kXAt = kXTr ? 2 : 4, kWAt = kWTr ? 1 : 4;
    uint32_t x_at[kXAt], w_at[kWAt];
    {
        const int l = lane_now(), half = l >> 5, r32 = l & 31, i16 = l & 15;
        const uint32_t base = (uint32_t)(uintptr_t)(LdsBytes)stages + ld.stage;
        const uint32_t row_at = r32 * 128 + ((half ^ swizzle(r32)) << 4);
        const uint32_t tr_at = (half * 8 + (i16 >> 2)) * 256 + ((l >> 4) & 1) * 32 + (i16 & 3) * 8;
#pragma unroll
        for (int i = 0; i < kXAt; ++i)
            x_at[i] = base + (kXTr ? tr_at + ((wm ^ (i16 >> 2) ^ (i * 2)) << 6) : (row_at ^ (i << 5)) + wm * 4096);
#pragma unroll
        for (int i = 0; i < kWAt; ++i)
            w_at[i] = base + (kWTr ? tr_at + ((wn ^ (i16 >> 2)) << 6) : (row_at ^ (i << 5)) + wn * 4096);
    }
    auto read_tr = [&](uint32_t at) { return read_transposed(at, at + 1024); };
    auto read_rows = [&](uint32_t at) -> bf16x8 { return *(LdsRows)(uintptr_t)at; };
    // rows (mt * 2 + wm) * 32 .. and columns (nt * 4 + wn) * 32 .. of the tile
    auto read_x = [&](int mt, int j) {
        if (mt >= A) return;
        if constexpr (kXTr) xf[mt][j] = read_tr(x_at[mt & 1] + (mt >> 1) * kHalf + j * 4096);
        else xf[mt][j] = read_rows(x_at[j] + (mt >> 1) * kHalf + (mt & 1) * 8192);
    };
    auto read_w = [&](int nt, int j) {
        if constexpr (kWTr) wf[nt][j] = read_tr(w_at[0] + (2 + nt) * kHalf + j * 4096);
        else wf[nt][j] = read_rows(w_at[j] + (2 + nt) * kHalf);
    };

    // The products of rows mt0, mt0 + 1 and columns nt, 16 sum indexes at a time, behind each `also(j)`.
    auto multiply = [&](int mt0, int nt, auto also) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            also(j);
#pragma unroll
            for (int mt = mt0; mt < mt0 + 2; ++mt)
                if (mt < A)
                    acc[nt][mt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[nt][j], xf[mt][j],
                                                                          acc[nt][mt], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr int kStores = O == to::kSwiglu ? 2 * A : O == to::kSwigluGrad || O == to::kF32 ? 8 * A : 4 * A;
    auto meet = [&]() {
        if (ld.stored > 0) {
            --ld.stored;
            meet_loaded<kLoads + kStores>();
        } else {
            meet_loaded<kLoads>();
        }
    };
    // One block. At each barrier what is read from then on has arrived, and what is loaded over has been
    // read.
    auto step = [&]() {
        const uint32_t cur = ld.stage;
        meet();
        multiply(0, 0, [&](int j) {
            read_w(1, j);
            read_x(2, j);
            if (j == 1) ld.template load<false>(stages, cur, 0);
        });
        multiply(0, 1, [&](int j) {
            read_x(3, j);
            if (j == 1) ld.template load<true>(stages, cur, 0);
        });
        ld.stage ^= kStage;
#pragma unroll
        for (int i = 0; i < kXAt; ++i) x_at[i] ^= kStage;
#pragma unroll
        for (int i = 0; i < kWAt; ++i) w_at[i] ^= kStage;
        meet();
        multiply(2, 0, [&](int j) {
            read_x(0, j);
            if (j == 1) ld.template load<true>(stages, cur, 1);
        });
        multiply(2, 1, [&](int j) {
            read_w(0, j);
            read_x(1, j);
            if (j == 1) ld.template load<false>(stages, cur, 1);
        });
        ld.advance();
    };

    // A product's 32 x 32 results: element i of a lane is column (i >> 2) * 8 + (lane >> 5) * 4 + (i & 3) of
    // row lane & 31. eight(): the lanes' halves trade, so that a lane has columns (2 * g + (lane >> 5)) * 8
    // .. of its row.
    auto eight = [](const f32x16 &v, int g, float (&to)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[g * 8 + i]),
                                                            __float_as_uint(v[g * 8 + 4 + i]), false, false);
            to[i] = __uint_as_float(s[0]);
            to[4 + i] = __uint_as_float(s[1]);
        }
    };
    auto eight_bf16 = [](const f32x16 &v, int g) {
        const auto s = __builtin_amdgcn_permlane32_swap(pair(v[g * 8], v[g * 8 + 1]),
                                                        pair(v[g * 8 + 4], v[g * 8 + 5]), false, false);
        const auto t = __builtin_amdgcn_permlane32_swap(pair(v[g * 8 + 2], v[g * 8 + 3]),
                                                        pair(v[g * 8 + 6], v[g * 8 + 7]), false, false);
        return u32x4{s[0], t[0], s[1], t[1]};
    };
    // Neighbouring groups of 16 lanes trade, so that a and b are of rows lane & 15 and 16 more, 64 bytes of
    // a row in four lanes; and back. (With 32 bytes of a row stored together L2 takes twice the
    // requests.)
    auto trade = [](u32x4 &a, u32x4 &b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto s = __builtin_amdgcn_permlane16_swap(a[i], b[i], false, false);
            a[i] = s[0];
            b[i] = s[1];
        }
    };
    // The tile's output. Every wavefront makes the same number of stores whatever the rows and columns
    // that are there, kStores at least: the waits for loads count past them.
    auto finish = [&](int tile) {
        const Tile t = ld.at(tile);
        const auto &p = argument();
        const int rows = t.rows;
        const size_t row0 = F == form::kWgrad ? (size_t)t.e * p.m + t.m0 : (size_t)t.row0;
        const int l = lane_now();
        const uint32_t r = wm * 32 + (l & 15);
        // a lane's columns of 32: eight of 16 bits, or four and four more of 32
        const uint32_t c16 = ((l >> 4) & 1) * 16 + (l >> 5) * 8, c32 = ((l >> 4) & 1) * 8 + (l >> 5) * 4;
        const uint32_t n = p.n;
        auto put_rows = [](const Rows &to, uint32_t off, uint32_t step, u32x4 a, u32x4 b) {
            to.put(off, a);
            to.put(off + step, b);
        };
        if constexpr (O == to::kSwiglu) {
            const uint32_t I = n / 2, c = t.nblk * 128 + wn * 32 + c16;
            const Rows h(p.out, row0, rows, I, 2);
#pragma unroll
            for (int mt = 0; mt < A; ++mt) {
                const uint32_t row = r + mt * 64;
                if (p.out2) {
                    const Rows gu(p.out2, row0, rows, n, 2);
                    const uint32_t off = c < I ? (row * n + c) * 2 : kNone;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        u32x4 a = eight_bf16(acc[nt][mt], 0), b = eight_bf16(acc[nt][mt], 1);
                        trade(a, b);
                        put_rows(gu, off + nt * I * 2, n * 32, a, b);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[0][mt][i] = swiglu(acc[0][mt][i], acc[1][mt][i]);
                u32x4 a = eight_bf16(acc[0][mt], 0), b = eight_bf16(acc[0][mt], 1);
                trade(a, b);
                put_rows(h, c < I ? (row * I + c) * 2 : kNone, I * 32, a, b);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            const Rows out(p.out, row0, rows, O == to::kSwigluGrad ? n * 2 : n, O == to::kF32 ? 4 : 2);
#pragma unroll
            for (int mt = 0; mt < A; ++mt)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const f32x16 &v = acc[nt][mt];
                    const uint32_t row = r + mt * 64, c0 = t.nblk * kTile + nt * 128 + wn * 32, c = c0 + c16;
                    const uint32_t off = c < n ? (row * n + c) * 2 : kNone;
                    if constexpr (O == to::kBf16) {
                        u32x4 a = eight_bf16(v, 0), b = eight_bf16(v, 1);
                        trade(a, b);
                        put_rows(out, off, n * 32, a, b);
                    } else if constexpr (O == to::kF32) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const uint32_t c = c0 + g * 16 + c32, at = c < n ? (row * n + c) * 4 : kNone;
                            u32x4 a{__float_as_uint(v[g * 8]), __float_as_uint(v[g * 8 + 1]),
                                    __float_as_uint(v[g * 8 + 2]), __float_as_uint(v[g * 8 + 3])};
                            u32x4 b{__float_as_uint(v[g * 8 + 4]), __float_as_uint(v[g * 8 + 5]),
                                    __float_as_uint(v[g * 8 + 6]), __float_as_uint(v[g * 8 + 7])};
                            trade(a, b);
                            if (p.accumulate) {
                                const f32x4 x = __builtin_bit_cast(f32x4, out.get(at));
                                const f32x4 y = __builtin_bit_cast(f32x4, out.get(at + n * 64));
                                a = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, a) + x);
                                b = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, b) + y);
                            }
                            put_rows(out, at, n * 64, a, b);
                        }
                    } else if constexpr (O == to::kSwigluGrad) {
                        const Rows gu(p.in, row0, rows, n * 2, 2);
                        const uint32_t at = off == kNone ? kNone : off + row * n * 2;
                        u32x4 gate[2] = {gu.get(at), gu.get(at + n * 64)};
                        u32x4 up[2] = {gu.get(at + n * 2), gu.get(at + n * 66)};
                        trade(gate[0], gate[1]);
                        trade(up[0], up[1]);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float d[8], a[8], b[8];
                            eight(v, g, d);
                            unpack8(gate[g], a);
                            unpack8(up[g], b);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float s = sigmoid(a[i]), du = d[i] * (a[i] * s);
                                a[i] = d[i] * b[i] * (s * __builtin_fmaf(a[i], 1.0f - s, 1.0f));
                                b[i] = du;
                            }
                            gate[g] = pack8(a);
                            up[g] = pack8(b);
                        }
                        trade(gate[0], gate[1]);
                        trade(up[0], up[1]);
                        put_rows(out, at, n * 64, gate[0], gate[1]);
                        put_rows(out, at + n * 2, n * 64, up[0], up[1]);
                    } else {
                        // z of eight columns, with the bias
                        auto z8 = [&](int g, float (&d)[8]) {
                            eight(v, g, d);
                            if (p.bias) {
                                float b[8];
                                const uint32_t at = (c0 + g * 16 + (l >> 5) * 8) * 2;
                                unpack8(Rows(p.bias, 0, 1, n, 2).get(at), b);
#pragma unroll
                                for (int i = 0; i < 8; ++i) d[i] += b[i];
                            }
                        };
                        float d[8];
                        u32x4 x[2];
                        if (p.out2) {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                z8(g, d);
                                x[g] = pack8(d);
                            }
                            trade(x[0], x[1]);
                            put_rows(Rows(p.out2, row0, rows, n, 2), off, n * 32, x[0], x[1]);
                        }
                        if (p.in) {
                            const Rows res(p.in, row0, rows, n, 2);
                            x[0] = res.get(off);
                            x[1] = res.get(off + n * 32);
                            trade(x[0], x[1]);
                        }
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            z8(g, d);
                            if (p.act != EP_ACT_NONE)
#pragma unroll
                                for (int i = 0; i < 8; ++i) d[i] = activate(p.act, d[i]);
                            if (p.in) {
                                float b[8];
                                unpack8(x[g], b);
#pragma unroll
                                for (int i = 0; i < 8; ++i) d[i] += b[i];
                            }
                            x[g] = pack8(d);
                        }
                        trade(x[0], x[1]);
                        put_rows(out, off, n * 32, x[0], x[1]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        clear();
        ld.stored = 3;
    };

#pragma unroll
    for (int j = 0; j < 4; ++j) {
        read_w(0, j);
        read_x(0, j);
        read_x(1, j);
    }
    clear();
    if (ld.parts < A) ld.stored = 0;           // the last tile made fewer stores than its kStores here
    ld.parts = A;
    for (; tile < end; ++tile) {
        for (int kb = ld.blocks_of(ld.at(tile)); kb > 0; --kb) step();
        finish(tile);
    }
}
#endif

template <int F, int O>
__global__ __launch_bounds__(kThreads) void product_kernel(Product p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    // aligned so that the stage is one bit of an address
    __shared__ __attribute__((aligned(kStage))) uint8_t stages[2 * kStage];
    __shared__ Tile list[kList];
    static_assert(sizeof(TileTable) <= sizeof(stages), "the table is done with before the first block");
    TileTable &table = *reinterpret_cast<TileTable *>(stages);
    const int n_tiles = (p.n + kTile - 1) / kTile, m_tiles = (p.m + kTile - 1) / kTile;
    // of each gridDim.x tiles in a row an XCD takes one eighth (its workgroups are blockIdx.x mod 8,
    // gridDim.x is a multiple of 8)
    const int slot = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    const int lane = threadIdx.x & (kWave - 1), grid = gridDim.x;
    for (int first = slot;;) {                 // kList tiles at a time
        int total;
        if constexpr (F == form::kWgrad) total = p.E * m_tiles * n_tiles;
        else total = build_table(table, p) * n_tiles;
        // The tiles of a last round that leaves at least half of the workgroups without one are cut, so
        // that each of them gets a piece.
        const int rest = total % grid, whole = total - rest;
        const int cuts = rest ? min(grid / rest, kTile / kPart) : 1;
        const int pieces = whole + rest * cuts;
        if (first >= pieces) break;
        const int tiles = min((pieces - first + grid - 1) / grid, kList);
        Tile mine{};
        if (lane < tiles) {
            int at = first + lane * grid, piece = 0;
            if (at >= whole && cuts > 1) {
                piece = (at - whole) % cuts;
                at = whole + (at - whole) / cuts;
            }
            int columns;                       // nothing of its divisions stays in registers
            asm volatile("" : "=s"(columns) : "0"(uniform(n_tiles)));
            if constexpr (F == form::kWgrad) mine = locate_wgrad(p, at, m_tiles, columns);
            else mine = locate(table, p, at, columns);
            if (first + lane * grid >= whole && cuts > 1) cut(mine, piece, cuts, F == form::kWgrad);
        }
        const int parts = (mine.rows + kPart - 1) / kPart;
        const uint64_t some = __ballot(parts > 0);
        uint64_t with[5];
#pragma unroll
        for (int a = 1; a <= 4; ++a) with[a] = __ballot(parts == a);
        if ((int)threadIdx.x < tiles) list[threadIdx.x] = mine;
        __syncthreads();                       // the list is there, the table is done with
        const int n_list = __popcll(some);     // a piece that is empty can only be the last
        if (n_list > 0) {
            Stream<F, O> ld(p, list, n_list);
            ld.start(stages);
            int tile = 0;
            auto run_some = [&](auto a) {      // the tiles from here on that have A parts
                constexpr int A = decltype(a)::value;
                if (tile == n_list) return;
                const uint64_t without = ~(with[A] >> tile);
                const int n = min(without ? (int)__builtin_ctzll(without) : kWave, n_list - tile);
                if (n > 0) run<F, O, A>(ld, stages, tile, tile + n);
                tile += n;
            };
            while (tile < n_list) {
                run_some(std::integral_constant<int, 4>{});
                run_some(std::integral_constant<int, 3>{});
                run_some(std::integral_constant<int, 2>{});
                run_some(std::integral_constant<int, 1>{});
            }
            meet_loaded<0>();                  // no direct load is left to write LDS
        }
        first += tiles * grid;
    }
#else
    (void)p;
#endif
}

bool no_rows(const Product &p) { return p.pairs == 0 || (p.offset && p.rows == 0); }

// One workgroup per CU, or as many as there can be pieces of tiles.
template <int F, int O>
hipError_t launch_product(const Product &p, hipStream_t stream)
{
    int64_t tiles = (p.n + kTile - 1) / kTile;
    if (F != form::kWgrad && no_rows(p)) return hipSuccess;
    if (F == form::kWgrad) {
        tiles *= (int64_t)p.E * ((p.m + kTile - 1) / kTile);
    } else {
        const int64_t experts = p.pairs < p.E ? p.pairs : p.E;
        tiles *= p.pairs / kTile + experts;
    }
    tiles *= kTile / kPart;
    const dim3 grid((unsigned)(tiles < kCus ? (tiles + 7) / 8 * 8 : kCus));
    return launch(product_kernel<F, O>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_expert_gemm(const Product &p, hipStream_t stream)
{
    if (!no_rows(p) && few_rows(p, false)) return launch_few_gemm(p, stream);
    return launch_product<form::kForward, to::kBf16>(p, stream);
}

hipError_t launch_expert_swiglu(const Product &p, hipStream_t stream)
{
    if (!no_rows(p) && few_rows(p, true)) return launch_few_swiglu(p, stream);
    return launch_product<form::kForward, to::kSwiglu>(p, stream);
}

hipError_t launch_expert_dgrad(const Product &p, hipStream_t stream)
{
    if (!no_rows(p) && few_dgrad(p)) return launch_few_dgrad(p, false, stream);
    return launch_product<form::kDgrad, to::kBf16>(p, stream);
}

hipError_t launch_expert_swiglu_dgrad(const Product &p, hipStream_t stream)
{
    if (!no_rows(p) && few_dgrad(p)) return launch_few_dgrad(p, true, stream);
    return launch_product<form::kDgrad, to::kSwigluGrad>(p, stream);
}

hipError_t launch_expert_wgrad(const Product &p, bool f32, hipStream_t stream)
{
    if (few_wgrad(p)) return launch_few_wgrad(p, f32, stream);
    return f32 ? launch_product<form::kWgrad, to::kF32>(p, stream)
               : launch_product<form::kWgrad, to::kBf16>(p, stream);
}

hipError_t launch_linear(const Product &p, hipStream_t stream)
{
    if (!no_rows(p) && few_rows(p, false)) return launch_few_linear(p, stream);
    return launch_product<form::kForward, to::kLinear>(p, stream);
}

}  // namespace ep
