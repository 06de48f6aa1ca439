// The barriers by which the prefix's issuing warps tell a tile's softmax warps
// that P V of a page is complete (shared_prefix.cu).  Host code too: a test
// walks through their phases.
//
// A wait by parity knows a phase only from the one before it and the one
// after: it may be made for page n when page n - PV_BARS is known to be complete and
// page n + PV_BARS cannot be yet.  A softmax warp waits for page n - 2 at every page
// n, and for page n - 1 where it rescales O, before it hands over page n, and for
// the last page at a tile's end.  So with two barriers in turn the page before on
// the same barrier was always waited for, and the page after is never handed
// over.  On a single one, "n - 1, then n" at a tile's end could meet P V of n already
// complete, and then waited for a phase of the next tile.  That S of page n is
// complete would tell of P V of page n - 2 as well, but only as long as commits arrive
// at two barriers in the order of their issue; the wait of its own costs nothing
// (the call of 64 requests x 16 tokens x 40 heads on 32768 positions: 550-555 us with
// it, 566 without).
#pragma once

#include <cstdint>

namespace dflash {

constexpr int PV_BARS = 2;
constexpr int pv_bar(int page) { return page % PV_BARS; }
constexpr uint32_t pv_phase(int page) { return static_cast<uint32_t>(page / PV_BARS); }

}  // namespace dflash
