// products_choice.h -- which kernel the products of E4M3 or bf16 rows take, by sizes, types
// and alignment.  The rule stands apart from the launches, in plain C++, so that it can be
// asked on a host what a product takes: a `launch` has
//   stream<MODE, NT, RT, TC, W>()              few rows, a block 16*RT channels x 8*TC rows
//   tiles<MODE, DMA, NB, WT, WN, FT, FN>()     tiles of 16*WT*FT rows x 16*WN*FN channels
//   groups<MODE, DMA>()                        groups' tiles of 64 to 256 rows x 256
// as the kernels of kernels_products.hip have them, and one of these is called.
#pragma once

#include <cstddef>
#include <cstdint>

namespace moe {

// how a stage is multiplied (kernels_products.hip)
enum { F8 = 0, F8X = 1, BF16 = 2 };

struct ProductSizes {
    int64_t M, N, K, E;                 // rows, channels, bytes of a row, experts
    bool copies;                        // rows that the load unit can copy into LDS
};

constexpr int64_t CUS = 256;

inline int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

constexpr int64_t NEAR = 1ll << 31;     // bytes from a buffer's beginning that lane offsets reach

// rows that the load unit can copy into LDS: on 4 bytes, and within reach.  `gathered`:
// how many rows x has where they are taken by number, else 0.
inline bool copies_rows(const void *x, const void *w, int64_t ldx, int64_t ldw, int64_t w_stride, int64_t gathered)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w);
    return at % 4 == 0 && ldx % 4 == 0 && ldw % 4 == 0 && w_stride % 4 == 0 && ldw <= NEAR / 256 &&
           ldx <= NEAR / (gathered ? gathered : 256);
}

// A tile's time: of a stage, of the rest, and what is added to a stage where the last
// round has a CU alone with one block.  Fitted to the times in kernels_products.hip and some
// 20 more.  On the 70 shapes of profiles/e4m3_product_kernels.csv the kernel that is taken,
// streams among them, loses to the fastest one 0.3 % on average and 14 % at most for bf16 outputs, 1.9 and
// 21 % for fp32; where rows pass through registers 0.7 and 11 %, 2.0 and 22 %.
struct TileCost {
    int bt, bn;
    double stage, fixed, alone;                      // us
};

// The tile whose rounds over the CUs cost least.
template <size_t N>
int cheapest(const TileCost (&c)[N], const ProductSizes &a)
{
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < (int)N; ++i) {
        const int64_t n = ceil_div(ceil_div(a.M, c[i].bt) * ceil_div(a.N, c[i].bn), CUS);
        const double stages = a.K / 128.0;
        const double cost = n * (c[i].stage * stages + c[i].fixed) + (n % 2 ? c[i].alone * stages : 0.0);
        if (i == 0 || cost < least) {
            best = i;
            least = cost;
        }
    }
    return best;
}

template <int MODE, typename Launch>
void choose_dense_tiles(const ProductSizes &a, Launch &launch)
{
    // Through registers, a piece crossing words and lines: 333 x 5003 x 2048 with 64x64 / 64x128 / 128x256
    // 18.1 / 19.0 / 30.6 us, 512 x 6144 x 6144 63 / 59 / 89, 4096 x 6144 x 6144 493 / 353 / 266 (copied
    // 140); fp32 outputs 22 / 23 / 46, 75 / 135 / 138 and 567 / 796 / 414.  256x256 has too few registers (477).
    if (!a.copies) {
        if constexpr (MODE == F8) {
            static constexpr TileCost cost[] = {{64, 64, 0.40, 1.5, 0.25}, {64, 128, 0.60, 2.0, 0.3}, {128, 256, 1.8, 4.0, 0.0}};
            switch (cheapest(cost, a)) {
            case 0: launch.template tiles<MODE, false, 2, 2, 2, 2, 2>(); break;
            case 1: launch.template tiles<MODE, false, 2, 2, 4, 2, 2>(); break;
            default: launch.template tiles<MODE, false, 2, 2, 4, 4, 4>(); break;
            }
        } else {
            static constexpr TileCost cost[] = {{64, 64, 0.46, 1.5, 0.2}, {128, 256, 2.8, 4.0, 0.0}};
            if (cheapest(cost, a) == 0)
                launch.template tiles<MODE, false, 2, 2, 2, 2, 2>();
            else
                launch.template tiles<MODE, false, 2, 2, 4, 4, 4>();
        }
        return;
    }
    if constexpr (MODE == F8) {
        static constexpr TileCost cost[] = {{64, 64, 0.253, 1.5, 0.08}, {64, 128, 0.36, 2.2, 0.0}, {128, 128, 0.56, 3.5, 0.0},
                                            {128, 256, 0.95, 4.0, 0.0}, {256, 256, 1.55, 7.0, 0.0}};
        switch (cheapest(cost, a)) {
        case 0: launch.template tiles<MODE, true, 4, 2, 2, 2, 2>(); break;
        case 1: launch.template tiles<MODE, true, 3, 2, 4, 2, 2>(); break;
        case 2: launch.template tiles<MODE, true, 3, 4, 2, 2, 4>(); break;
        case 3: launch.template tiles<MODE, true, 3, 2, 4, 4, 4>(); break;
        default: launch.template tiles<MODE, true, 2, 2, 4, 8, 4>(); break;
        }
    } else {
        static constexpr TileCost cost[] = {{64, 64, 0.305, 1.5, 0.2}, {64, 128, 0.52, 2.5, 0.2}, {128, 128, 1.02, 3.5, 0.0},
                                            {128, 256, 1.65, 4.0, 0.0}};
        switch (cheapest(cost, a)) {
        case 0: launch.template tiles<MODE, true, 4, 2, 2, 2, 2>(); break;
        case 1: launch.template tiles<MODE, true, 3, 2, 4, 2, 2>(); break;
        case 2: launch.template tiles<MODE, true, 3, 4, 2, 2, 4>(); break;
        default: launch.template tiles<MODE, true, 3, 2, 4, 4, 4>(); break;
        }
    }
}

// Streams as long as their blocks fit the card: a block has its K in W parts at once, where
// a tile's stages come one after the other at 0.45 us each (64 x 6144 x 6144: stream 11.9 us,
// tile 21.8; 256 x 2048 x 7168 12.7 and 24.9; 64 x 4096 x 7168 9.0 and 22.9; of fp32
// 64 x 6144 x 6144 14.2 and 28.4).  With half as many blocks again they are near each other
// (128 x 6144 x 2048 9.3 and 9.0; 128 x 6144 x 6144 19.2 and 21.9, of fp32 22.1 and 28.6), with
// more the tiles win (256 x 6144 x 6144 29.5 and 25.7).  Where rows are not copied the tiles take
// twice as long, the streams half as much again (128 x 6144 x 6144 32.4 and 44.7, 256 rows 48.3
// and 46.0; of fp32 256 rows 51.0 and 67.9), so they go on to 2 or 3 blocks for each CU.
// Smaller blocks while they fit: of 16 channels, 32, then 64 (64 x 4096 x 7168:
// 12.7, 9.0, 11.7; 48 x 2048 x 7168 of F8X: 7.9, 10.0), of 8 rows if there are no more; 16
// waves where they alone fill the card (1 x 2048 x 7168 4.5 us, 8 waves 4.8; 1 x 6144 x 6144
// 8.0 and 7.0).  Up to 32 rows all are streams (32 x 24576 x 6144 24.8, tiles 24.6; 32 x 8192 x
// 7168 11.5 and 24.2).
template <int MODE, int TILE_MODE, typename Launch>
void choose_dense(const ProductSizes &a, Launch &launch)
{
    const auto blocks = [&](int t, int n) { return ceil_div(a.M, t) * ceil_div(a.N, n); };
    if (a.M <= 8) {
        if (blocks(8, 16) <= CUS)
            launch.template stream<MODE, false, 1, 1, 16>();
        else
            launch.template stream<MODE, false, 1, 1, 8>();
    } else if (a.M <= 16) {
        if (blocks(16, 16) <= CUS)
            launch.template stream<MODE, false, 1, 2, 8>();
        else
            launch.template stream<MODE, false, 2, 2, 8>();
    } else if (a.M <= 32) {
        if (blocks(32, 16) <= CUS)
            launch.template stream<MODE, false, 1, 4, 8>();
        else if (blocks(32, 32) <= CUS)
            launch.template stream<MODE, false, 2, 4, 8>();
        else
            launch.template stream<MODE, false, 2, 4, 4>();
    } else if (blocks(32, 16) <= CUS) {
        launch.template stream<TILE_MODE, false, 1, 4, 8>();
    } else if (blocks(32, 32) <= CUS) {
        launch.template stream<TILE_MODE, false, 2, 4, 8>();
    } else if (2 * blocks(32, 64) <= CUS * (a.copies ? (TILE_MODE == F8 ? 2 : 3) : (TILE_MODE == F8 ? 4 : 6))) {
        launch.template stream<TILE_MODE, false, 4, 4, 4>();
    } else {
        choose_dense_tiles<TILE_MODE>(a, launch);
    }
}

// Few blocks in all, as a router's logits are: whatever the groups' sizes, K in eight parts.
// 64 rows in 2 groups of 256 x 6144 of bf16 6.2 us (tiles 32, 16-row streams 8.9), 128 rows 6.9 in
// blocks of 16 rows and 8.7 of 8, 1000 rows 14.5 (tiles 34); 100 x 4 of 8 of 512 x 4096
// 7.8 (tiles 16.8).  False where there are more.
template <int MODE, typename Launch>
bool choose_few(const ProductSizes &a, int64_t rows, Launch &launch)
{
    const auto blocks = [&](int t, int n) { return (a.E < a.M ? a.E : a.M) * ceil_div(rows, t) * ceil_div(a.N, n); };
    if (blocks(8, 16) <= CUS / 2)
        launch.template stream<MODE, false, 1, 1, 8>();
    else if (blocks(16, 16) <= CUS)
        launch.template stream<MODE, false, 1, 2, 8>();
    else if (blocks(32, 32) <= CUS)
        launch.template stream<MODE, false, 2, 4, 8>();
    else
        return false;
    return true;
}

// By the rows of a group on average, with borders from weights of 2048 x 2048 and 4096 x 6144.
// Streams up to 12 (24 where tiles have the bf16 unit too):
// E4M3, 64 experts of 2048 x 2048 with 16 rows each 44.9 us and tiles 41.5, of bf16 105.8 and
// 114.5, 24 rows 115 and 123, 32 rows 117.6 and 117.0.  Weights that pass the caches are read
// so too: 256 of 4096 x 6144 by 16 tokens x 8 280 us and 317, by 256 tokens 897 and 938;
// where they stay in them not: 64 of 2048 x 2048 by 64 tokens 48 and 40.
// Tiles: 64 x 128 below 24 rows (bf16 64: 125 rows 157 us, groups' tiles 151, 32 rows
// 116 and 146) and where the groups' do not fill the card (16 experts of 2048 x 4096, 64 rows each
// 28 us, groups' 47; 512 rows each 125 and 107).  F8X: 64 x 128 below 128 rows (125
// rows 123 us, 128 x 256 136; 512 rows 402 and 312).  Rows that are not copied (64 experts of
// 2048 x 2048): E4M3 64 x 128 below 256 rows (125 rows 160 us, 128 x 256 170; 512 rows 481 and 373); on
// the bf16 unit streams up to 64 (32 rows 97, 128 x 256 123; 64 rows 167 and 181; of bf16 236 and the
// groups' tiles 277), then F8X 128 x 256, bf16 the groups' tiles (125 rows 290, 128 x 256 338).
template <int MODE, int TILE_MODE, typename Launch>
void choose_grouped(const ProductSizes &a, Launch &launch)
{
    const int64_t rows = ceil_div(a.M, a.E);
    if (rows <= 12 ? choose_few<MODE>(a, rows, launch) : choose_few<TILE_MODE>(a, rows, launch))
        return;
    // weights that the last-level cache does not keep from one call to the next, and
    // that hardly anyone reads twice
    const bool passing = (int64_t)(a.E < a.M ? a.E : a.M) * a.N * a.K >= (512ll << 20);
    if (rows <= 4) {
        if (passing)
            launch.template stream<MODE, true, 2, 2, 4>();
        else
            launch.template stream<MODE, false, 2, 2, 4>();
    } else if (rows <= (TILE_MODE == F8 ? 12 : a.copies ? 24 : 64)) {
        if (passing && rows <= 12)
            launch.template stream<MODE, true, 4, 4, 4>();
        else
            launch.template stream<MODE, false, 4, 4, 4>();
    } else if (!a.copies) {
        if constexpr (TILE_MODE == BF16)
            launch.template groups<BF16, false>();
        else if (TILE_MODE == F8 && rows < 256)
            launch.template tiles<TILE_MODE, false, 2, 2, 4, 2, 2>();
        else
            launch.template tiles<TILE_MODE, false, 2, 2, 4, 4, 4>();
    } else if constexpr (TILE_MODE == F8X) {
        if (rows < 128)
            launch.template tiles<F8X, true, 3, 2, 4, 2, 2>();
        else
            launch.template tiles<F8X, true, 3, 2, 4, 4, 4>();
    } else {
        if (rows < (TILE_MODE == BF16 ? 64 : 24) || a.E * ceil_div(rows, 256) * ceil_div(a.N, 256) < CUS)
            launch.template tiles<TILE_MODE, true, 3, 2, 4, 2, 2>();
        else
            launch.template groups<TILE_MODE, true>();
    }
}

}  // namespace moe
