// How the blocks of a grouped launch find their tile (device side).
#pragma once
#include "launch.hpp"

namespace moe {
namespace {

// Which (M tile, N tile) pair a block computes.  Blocks go to the eight
// XCDs round robin (block b runs on XCD b % 8), so block b takes logical
// slot (b % 8) * per + b / 8: each XCD walks one contiguous stretch of the
// logical order.  That order is: runs of tiles that share weights (one
// expert, or up to 8 dense row tiles), inside a run N tile by N tile with
// the M tile fastest.  A run of `cnt` tiles starting at tile `first`
// occupies slots [first*ntn, (first+cnt)*ntn), so slot / ntn names a tile of
// the run that owns the slot.  With a tile table the routed slots and the
// shared-expert slots (the table's tail) are split across the XCDs
// separately, each XCD walking a stretch of either: the shared tiles re-read
// one weight matrix per run and would otherwise all land on the last XCD.
// The grid holds 8 * (per_routed + per_shared) blocks or more (launch
// grids carry 16 spare blocks).  Returns false for blocks without work.
struct Job {
    int gi, expert, row0, rows, n0;
};

// xcd_slot_pair with the shared stretch of an XCD before its routed one.
__device__ __forceinline__ int xcd_slot_pair_shared_first(int b, int total_r, int total) {
    const int per = (total_r + 7) >> 3, per_s = (total - total_r + 7) >> 3;
    const int slot = b >> 3, xcd = b & 7;
    if (slot < per_s) {
        const int lin = total_r + xcd * per_s + slot;
        return lin < total ? lin : -1;
    }
    const int k = slot - per_s, lin = xcd * per + k;
    return (k < per && lin < total_r) ? lin : -1;
}

// With a tile table, BM is the table's rows per tile (the planner builds the
// table for the kernels that walk it), and the job comes from one load of
// the entry at slot / ntn, whose run fields place every tile of its run;
// the two tile counts come in one load.  Up to `shared_first` shared pairs go
// before the routed ones (for launches whose shared pairs take longer: the
// short ones then end the launch).
template <int BM, int BNO>
__device__ __forceinline__ bool pick_job(const GemmArgs& a, Job& jb, int shared_first = 0) {
    int total, total_r;  // active (M, N) tile pairs, and the routed ones among them
    if (a.tiles) {
        const int2 nt = *reinterpret_cast<const int2*>(a.ntiles);
        total = nt.x * a.ntn;
        total_r = nt.y * a.ntn;
    } else {
        total = total_r = ((a.M + BM - 1) / BM) * a.ntn;
    }
    const int b = static_cast<int>(blockIdx.x);
    const int lin = total - total_r <= shared_first ? xcd_slot_pair_shared_first(b, total_r, total)
                                                    : xcd_slot_pair(b, total_r, total);
    if (lin < 0) return false;
    if (a.tiles) {
        const TileInfo t0 = a.tiles[lin / a.ntn];
        const int u = lin - t0.first * a.ntn, i = u % t0.count;
        jb.gi = t0.group;
        jb.expert = t0.expert;
        jb.row0 = t0.run_row0 + i * BM;
        jb.rows = min(BM, t0.run_rows - i * BM);
        jb.n0 = (u / t0.count) * BNO;
    } else {
        const int mtiles = total / a.ntn;
        const int first = (lin / a.ntn) & ~7, cnt = min(8, mtiles - first);
        const int u = lin - first * a.ntn;
        jb.gi = 0;
        jb.expert = 0;
        jb.row0 = (first + u % cnt) * BM;
        jb.rows = min(BM, a.M - jb.row0);
        if (jb.rows <= 0) return false;
        jb.n0 = (u / cnt) * BNO;
    }
    return jb.n0 < (jb.gi ? a.g[1].N : a.g[0].N);
}

}  // namespace
}  // namespace moe
