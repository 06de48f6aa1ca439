// The barriers by which the prefix's issuing warps tell a tile's softmax warps
// that P V of a page is complete (shared_prefix.cu).  Host code too: a test
// walks through their phases.
//
// A wait by parity knows a phase only from the one before it and the one
// after: it may be made for page n when page n - PV_BARS is known to be complete and
// page n + PV_BARS cannot be yet.  A softmax warp waits for page n's P V either before
// it hands over page n + 1, or at a tile's end, when n was the last page.  S of
// page n is complete by then and was issued behind P V of page n - 2, so with two
// barriers in turn both hold.  On a single one, "n - 1, then n" at a tile's end could
// meet P V of n already complete, and then waited for a phase of the next tile.
#pragma once

#include <cstdint>

namespace dflash {

constexpr int PV_BARS = 2;
constexpr int pv_bar(int page) { return page % PV_BARS; }
constexpr uint32_t pv_phase(int page) { return static_cast<uint32_t>(page / PV_BARS); }

}  // namespace dflash
