// How the router's rows are cut into blocks: host arithmetic alone, so that it can be
// compiled and tested without CUDA.
#pragma once

#include <algorithm>

#include <stdint.h>

namespace fc {

#define FC_ROUTER_WARPS 4   // of a block at most: of small blocks an SM takes nearly as many as another
#define FC_ROUTER_JOIN 8    // blocks of a cluster

struct RouterShape {
    int64_t sequences, tokens;  // rows = sequences * tokens
    int experts, k;
    int64_t groups;             // of rows that are balanced by themselves: 1 or sequences
    bool normalise;
};

struct RouterCut {
    int parts;  // blocks a group
    int rows;   // rows of a warp at a time
    int warps;  // of a block
    bool joins; // the grid is one cluster, which joins all
};

// Most blocks a group.
inline int64_t router_parts(int64_t sequences, int64_t tokens, int64_t groups)
{
    if (sequences * tokens == 0) return 1;
    return std::min<int64_t>(sequences * tokens / groups, std::max<int64_t>(1, 1216 / groups));
}

// How to cut the rows: as many of a warp at a time as leave the SMs' warps about the same
// number of tiles each, counting the instructions of a tile (some for each set of rows
// side by side, some for each tile) and what a tile waits for, in cycles.  `bytes` says
// what a block of `warps` warps with `rows` rows each needs of shared memory.
template <class F>
RouterCut router_cut(const RouterShape &n, int beside, int blocks, int step, int each, int tile, F bytes)
{
    const int64_t per = n.sequences * n.tokens / n.groups;
    const int64_t most = router_parts(n.sequences, n.tokens, n.groups);
    RouterCut best = {};
    double least = 0;
    for (int rows = 32; rows >= step; rows -= step) {  // whole steps: no tests of the rows
        RouterCut c = {};
        c.rows = rows;
        c.warps = FC_ROUTER_WARPS;
        while (c.warps > 1 && (per <= (int64_t)rows * (c.warps / 2) || bytes(c.warps, rows) > 110 * 1024))
            c.warps /= 2;
        const int64_t fit = 232448 / (int64_t)(bytes(c.warps, rows) + 1024);
        const int64_t slots = 152 * std::min<int64_t>(fit, blocks * FC_ROUTER_WARPS / c.warps) * c.warps;
        const int64_t tiles = n.groups * ((per + rows - 1) / rows);
        int64_t rounds = std::max<int64_t>(1, (tiles + slots - 1) / slots);  // no rows: no tiles
        const int64_t parts = (per + rows * c.warps * rounds - 1) / (rows * c.warps * rounds);
        c.parts = (int)std::max<int64_t>(1, std::min(parts, most));
        rounds = (per + (int64_t)rows * c.warps * c.parts - 1) / ((int64_t)rows * c.warps * c.parts);
        const int64_t an_sm = (std::min(n.groups * c.parts * c.warps, slots) + 151) / 152;
        const double sets = (rows + beside - 1) / beside;
        const double issue = rounds * an_sm * (each * sets + tile) / 4;
        const double wait = rounds * (200 * sets + 4 * tile + 1000);
        const double cost = std::max(issue, wait) + .3 * std::min(issue, wait);
        if (best.rows == 0 || cost < least) {
            least = cost;
            best = c;
        }
    }
    best.joins = n.groups * best.parts <= FC_ROUTER_JOIN;
    return best;
}

}  // namespace fc
