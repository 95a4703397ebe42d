// scan_window_phases.h -- which barrier, and which of its phases, announces dS of
// key tile u in the queries' backward kernel. Plain C++, so that the order of the
// roles can be checked on the host for every interleaving.
#pragma once

namespace scan {

// Two warps wait for dS of tile u: the one that issues dq += dS k, and the one that
// issues the next dP. A wait tells phases apart only by parity, and the softmax warps
// make dS(u + 1) without the first of the two: S(u + 1) is issued a tile earlier. On one
// barrier it could find that phase u had come and gone twice over. On two, the next
// phase of a tile's barrier is dS(u + 2), which needs S(u + 2), and that warp issues it
// after its wait.
constexpr int kDsBarriers = 2;
constexpr int ds_barrier(int u) { return u & 1; }
constexpr int ds_parity(int u) { return (u >> 1) & 1; }

}  // namespace scan
