// How products grouped by segment are cut into tiles, for the experts' products (experts.hip,
// mx.hip): a workgroup's tile, the segment it lies in, and the launches that make all of
// them. Not part of the ABI.
#pragma once

#include "experts.h"
#include "rows.h"

namespace moonep {
namespace segments {

using namespace rows;

// Sum of v over lanes 0 .. l, in every lane l: shifts within rows of 16 lanes, then each
// row's last lane into the rows behind it.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}

__device__ __forceinline__ int wave_scan(int v) {
    v = dpp_add<0x111, 0xf>(v);  // row_shr:1
    v = dpp_add<0x112, 0xf>(v);  // row_shr:2
    v = dpp_add<0x114, 0xf>(v);  // row_shr:4
    v = dpp_add<0x118, 0xf>(v);  // row_shr:8
    v = dpp_add<0x142, 0xa>(v);  // row_bcast:15
    v = dpp_add<0x143, 0xc>(v);  // row_bcast:31
    return v;
}

struct Tile {
    int seg, row, rows;  // segment (-1: none), first row on the rank, rows
};

// Tile `want` of a rank whose segments are cut into tiles of at most `bm` rows.
// Offsets are clamped to the rank's rows and the tile to its segment, so no table leads out
// of the arrays; a segment whose end is not past its start is empty.
__device__ __forceinline__ Tile find_tile(const int32_t *ptr, int n, int SK, int bm, int want) {
    int base = 0;
    for (int s = 0; s < n; s += 64) {
        const int j = s + lane_id();
        int lo = 0, len = 0;
        if (j < n) {
            lo = ptr[j];
            const int hi = min(ptr[j + 1], SK);
            len = lo >= 0 && hi > lo ? hi - lo : 0;
        }
        const int tiles = len > 0 ? (len - 1) / bm + 1 : 0;
        const int upto = wave_scan(tiles);
        const int total = readlane_i(upto, 63);
        if (want < base + total) {
            const int l = __ffsll((unsigned long long)__ballot(base + upto > want)) - 1;
            const int first = (want - base - (readlane_i(upto, l) - readlane_i(tiles, l))) * bm;
            const int rows = readlane_i(len, l);
            if (l < 0 || first < 0 || first >= rows) break;  // counts that overlap past 2^31
            return {s + l, readlane_i(lo, l) + first, min(bm, rows - first)};
        }
        base += total;
    }
    return {-1, 0, 0};
}

// Which tile a workgroup makes. The tiles are `units` (ranks, or segments) of tiles_m x
// tiles_n, cut into blocks. Workgroups go round the 8 XCDs in turn, each with an L2 of its
// own, so a block's tiles, which share their operands, go to one of them. Where units come in
// eighths each XCD takes whole ones, block by block; other numbers are dealt out by blocks.
// Within a block the columns are counted first: tiles of the same rows start next to one
// another and stay in step, so their rows come from HBM once (rows first: the decode shape,
// of two columns of tiles, read 10.6 GB in place of 9.4 and took 1.81 ms in place of 1.74). And the empty
// rows of tiles that end a rank then come in runs: dealt out one by one between the others,
// they fell on the same parts of the chip every time (31 ranks of 4 rows, 304 -> 5680 columns:
// 61 us in place of 37; a few full rows lose by it, one token a rank 43 to 45).
struct Order {
    uint32_t units, tiles_m, tiles_n;
    uint32_t block_m, block_n;    // tiles of a block
    uint32_t blocks_m, blocks_n;  // blocks of a unit
    uint32_t whole;               // each XCD takes whole units
    uint32_t each;  // tiles of each XCD, those that only fill up a block among them
};

struct Place {
    int unit, m, n;  // unit -1: none
};

__device__ __forceinline__ Place place(const Order &o, uint32_t first) {
    const uint32_t at = first + blockIdx.x / 8, xcd = blockIdx.x % 8;
    const uint32_t tiles = o.block_m * o.block_n, blocks = o.blocks_m * o.blocks_n;
    const uint32_t mine = at / tiles, in = at - mine * tiles;
    const uint32_t block = o.whole ? mine + xcd * (o.units / 8) * blocks : mine * 8 + xcd;
    const uint32_t unit = block / blocks, b = block - unit * blocks, bm = b / o.blocks_n;
    const uint32_t m_in = in / o.block_n;
    const uint32_t m = bm * o.block_m + m_in;
    const uint32_t n = (b - bm * o.blocks_n) * o.block_n + in - m_in * o.block_n;
    if (at >= o.each || unit >= o.units || m >= o.tiles_m || n >= o.tiles_n) return {-1, 0, 0};
    return {(int)unit, (int)m, (int)n};
}

// Launches one workgroup for each tile, in pieces a grid can hold. Blocks are of 32 tiles,
// what one XCD works on at a time, or of fewer where those would be too few to go round the
// XCDs evenly: 8 rows of 4 tiles for the products (1 or 2 rows: 0-15% slower; 4: 1%) and 4 of 8
// for the weight gradients (8: 3% slower with 56 experts a rank, 0-3% with fewer; 16: 1-8%).
template <typename F>
hipError_t in_order(int64_t units, int64_t tiles_m, int64_t tiles_n, int band, bool whole,
                    F &&launch) {
    int64_t most_m = band, most_n = 32 / band;
    auto parts = [](int64_t n, int64_t most) { return (n + most - 1) / most; };
    if (!whole)
        while (most_m * most_n > 1 && units * parts(tiles_m, most_m) * parts(tiles_n, most_n) < 64)
            most_m > most_n ? most_m /= 2 : most_n /= 2;
    const int64_t blocks_m = parts(tiles_m, most_m), blocks_n = parts(tiles_n, most_n);
    // of even size, so that few tiles only fill up
    const int64_t block_m = parts(tiles_m, blocks_m), block_n = parts(tiles_n, blocks_n);
    const int64_t all = units * blocks_m * blocks_n, tiles = block_m * block_n;
    if (all >= ((int64_t)1 << 31) / tiles) return hipErrorInvalidValue;  // no memory holds them
    Order o;
    o.units = (uint32_t)units;
    o.tiles_m = (uint32_t)tiles_m;
    o.tiles_n = (uint32_t)tiles_n;
    o.block_m = (uint32_t)block_m;
    o.block_n = (uint32_t)block_n;
    o.blocks_m = (uint32_t)blocks_m;
    o.blocks_n = (uint32_t)blocks_n;
    o.whole = whole;
    o.each = (uint32_t)((whole ? all / 8 : (all + 7) / 8) * tiles);
    constexpr uint32_t kPiece = 1u << 19;  // of each XCD's
    for (uint32_t at = 0; at < o.each; at += kPiece) {
        const uint32_t n = o.each - at < kPiece ? o.each - at : kPiece;
        launch(o, at, dim3(n * 8));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Most tiles of bm rows that the segments of one rank make: a segment of l > 0 rows makes
// at most (l - 1) / bm + 1.
inline int64_t most_tiles(const ExpertShape &sh, int bm) {
    const int64_t segs = sh.G + sh.B < sh.SK ? sh.G + sh.B : sh.SK;
    return (sh.SK - segs) / bm + segs;
}

inline int64_t tiles_of(int64_t n, int b) { return (n + b - 1) / b; }

// Tiles wanted at the least: fewer leave compute units without work.
constexpr int64_t kCus = 256, kFill = 192;

// Whether tiles that take a compute unit each leave at most a quarter of the units idle in
// their rounds. 525 tiles of 256x256 (three rounds, 68%) take 65 us where 128x128 takes 51.
inline bool fills(int64_t tiles) { return 4 * tiles >= 3 * kCus * ((tiles + kCus - 1) / kCus); }

}  // namespace segments
}  // namespace moonep
