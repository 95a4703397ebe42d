// scan_cross_phases.h -- how many places the rings of copies of attention to another
// sequence have, for heads of up to 64 and up to 128. Plain C++, so that the order of the
// kernels' roles can be checked on the host for every interleaving: a wait tells a
// barrier's phases apart only by parity, and whether that suffices depends on these
// numbers.
#pragma once

namespace scan {

constexpr int fwd_slots(int DP) { return DP == 128 ? 5 : 8; }  // tiles of keys and of values by turns
constexpr int bwd_slots(int DP) { return DP == 128 ? 5 : 8; }  // either backward kernel's, of two operands by turns
// Keys and values together. An even number: two groups of warps take them by turns, and
// a group that saw only every second phase of a place would take a phase that is to
// come for one that was.
constexpr int step_stages(int DP) { return DP == 128 ? 6 : 12; }

}  // namespace scan
