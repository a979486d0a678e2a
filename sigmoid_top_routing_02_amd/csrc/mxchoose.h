// Which kernel takes a grouped MXFP4 product, and the few-row kernels' grids.
#pragma once

#include <math.h>
#include <stdint.h>

namespace moe {

constexpr int MX_TILE_COLS = 256;                        // columns of B of a tile

enum MxKernel { ROWS16_NARROW, ROWS16, ROWS32, ROWS64, TILES };

// A few-row kernel's rows of A and column tiles (16 rows of B each) to a block.
struct MxRows { int high, tiles; };
constexpr MxRows mx_rows(MxKernel k) {
    return k == ROWS16_NARROW ? MxRows{16, 2} : k == ROWS16 ? MxRows{16, 4} : k == ROWS32 ? MxRows{32, 4} : MxRows{64, 4};
}

// Its grid: a row for each tile of rows, as the kernel deals them.
struct MxGrid { int64_t x, y; };
inline MxGrid mx_rows_grid(MxRows r, int64_t M, int G, int N) {
    const int wide = r.tiles * 16;
    return {((int64_t)N + wide - 1) / wide, M < G ? M : G + M / r.high};
}

// Whether it can be launched: a launch is held under the 2^32 threads that HIP
// documents, and a few-row kernel under 65535 grid rows for tiles of 16 rows.
inline bool mx_launches(MxRows r, int64_t M, int G, int N) {
    const MxGrid g = mx_rows_grid(r, M, G, N);
    return G + M / 16 <= 65535 && g.x * g.y * 256 <= 0xFFFFFFFFll;
}

// Which kernel: the one that the times below (us) make the fastest.  They were
// fitted to 445 measured calls, 1 to 256 groups of 1 to 4096 rows, even and skewed,
// N = 256 to 14336, K = 1024 to 32768, weights from HBM and from the caches; the choice
// costs 1.4 % over the fastest kernel on the average and 37 % at most.  The host
// knows the groups' sizes on the average only, and all groups of those calls had rows
// (but for a few of the skewed ones): where most are empty a large group goes to a
// kernel for few rows, which takes B once per row tile.  4 of 256 groups with 512
// rows each, N = 4096, K = 2048: 105 us, 21 without the empty ones; 16 with 256 rows
// 140 and 32.  A caller that knows such groups leaves them out.  c is the number of
// 512-value chunks of K; a round is a block (a tile) on every CU, and a call's last
// round counts whole while there are few of them.
//   16 rows, 2 column tiles: 3.8 + 0.4 c a round     16 rows, 4: 4.2 + 0.69 c
//   32 rows, 4 column tiles: 3.8 + 0.8 c             64 rows, 4: 4 + 1.19 c
//   whole tiles: 8.8 + 1.8 c up to 8.8 + 3.3 c when the round is full
//   half tiles:  8.8 + 2.4 c,   to 8.8 + 2.2 c
// and none takes less than B does from HBM at 5.5 TB/s, beside which a twentieth of
// the work shows.  Measured, in the order 16 x 2, 16 x 4, 32 x 4, 64 x 4, tiles:
// 32 groups, N = 4096, K = 7168: of 8 rows 103, 88, 90, 110, 107; of 32 rows 244, 202,
// 115, 129, 112; of 256 rows 1305, 1075, 670, 541, 160.  8 such groups of 32 rows: 52,
// 47, 24, 30, 38.  One group of N = 7168, K = 16384: 16 rows 17, 25, 26, 29, 63; 48
// rows 43, 47, 30, 36, 65; 128 rows 95, 90, 57, 39, 67.
inline MxKernel mx_choose(int64_t M, int G, int N, int K, int cus) {
    const double c = (double)((K + 511) / 512), groups = (double)(G < M ? G : M);
    const double mean = (double)M / groups;
    const double hbm = groups * N * K / 2 / 5.5e6;
    // row tiles of `high` rows: a group ends in half a tile on the average
    auto row_tiles = [&](int high) {
        if (groups == 1.0) return ceil(mean / high);
        return mean <= 0.68 * high ? groups : (double)M / high + 0.5 * groups;
    };
    auto beside = [&](double work) { return work > hbm ? work + 0.05 * hbm : hbm + 0.05 * work; };
    auto rows = [&](MxKernel k, double at, double per) {
        const MxRows r = mx_rows(k);
        const double rounds = row_tiles(r.high) * (double)mx_rows_grid(r, M, G, N).x / cus;
        return at + beside(per * c * (rounds < 4.0 ? ceil(rounds) : rounds));
    };
    auto tiles = [&](int high, double low, double full) {
        const double rounds = row_tiles(high) * ((N + MX_TILE_COLS - 1) / MX_TILE_COLS) / cus;
        return 8.8 + beside(rounds <= 1.0 ? (low + (full - low) * rounds) * c : ceil(rounds) * (8.8 + full * c) - 8.8);
    };
    const double halves = tiles(128, 2.4, 2.2), wholes = tiles(256, 1.8, 3.3);
    const double t[5] = {rows(ROWS16_NARROW, 3.8, 0.4), rows(ROWS16, 4.2, 0.69), rows(ROWS32, 3.8, 0.8),
                         rows(ROWS64, 4.0, 1.19), halves < wholes ? halves : wholes};
    int best = TILES;                                    // takes any size
    for (int i = TILES - 1; i >= 0; --i)
        if (t[i] <= t[best] && mx_launches(mx_rows((MxKernel)i), M, G, N)) best = i;
    return (MxKernel)best;
}

}  // namespace moe
