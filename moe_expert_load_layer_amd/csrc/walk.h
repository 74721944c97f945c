// Which tiles a workgroup of the 8-bit grouped product takes, and when it looks
// for the next one.  Plain arithmetic, so that it can be checked on a host.
#pragma once

#include <stdint.h>

namespace ep {

// The workgroups of one XCD (consecutive ones go round the 8 XCDs) share
// consecutive tiles: workgroup `block` of `blocks`, a multiple of 8, takes the
// tiles at, at + stride, ... below `to`.
struct TileWalk {
    int64_t at, to, stride;
};

constexpr TileWalk tile_walk(int64_t tiles, uint32_t block, uint32_t blocks) {
    const int64_t per = (tiles + 7) / 8, from = block % 8 * per, end = from + per;
    return TileWalk{from + block / 8, end < tiles ? end : tiles, (int64_t)blocks / 8};
}

// The step of a tile (of `steps`, with a ring of `stages`) before which a chained
// workgroup finds its next tile: its scales are loaded 4 steps before its rows.
constexpr int find_step(int steps, int stages) { return steps - stages - 4; }

// Whether a workgroup's tiles are chained, the next one's first loads among the
// last steps of this one.  Finding the next tile writes over what the stores of
// the tile before read, so at least one step's barrier has to lie between.
// Otherwise every tile starts afresh.
constexpr bool tiles_chained(int steps, int stages) { return find_step(steps, stages) > 0; }

// Workgroups that give each of m rows' tiles its own, where every group may end
// in a part tile.  Groups that overlap have more tiles than that.
constexpr int64_t tile_blocks(int64_t m, int64_t groups, int64_t n, int rows, int columns) {
    return ((m / rows + groups) * ((n + columns - 1) / columns) + 7) / 8 * 8;
}

}  // namespace ep
