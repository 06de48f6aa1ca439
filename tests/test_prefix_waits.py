"""The waits of the prefix's softmax warps for P V of a page, on the host: the
barrier and phase of each page as csrc/pv_done.h gives them, walked through with
P V completing as early and as late as the hand-overs between the warps allow.

A barrier's phase number is the count of completions so far; a wait by parity
for phase f passes where the count's parity is not f's."""
import itertools
import os
import shutil
import subprocess

import pytest

from block_diffusion_drafter_context_gb300.build import CSRC

PROGRAM = """
#include <cstdio>
#include "pv_done.h"
int main() {
  for (int n = 0; n < 64; ++n) std::printf("%d %u\\n", dflash::pv_bar(n), dflash::pv_phase(n));
}
"""


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    """(barrier, phase) of page n."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("pv")
    src, exe = os.path.join(d, "a.cpp"), os.path.join(d, "a")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", CSRC, src, "-o", exe], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    return [tuple(int(x) for x in line.split()) for line in lines if line]


def faults(place, at_end, tiles):
    """What can go wrong over tiles of so many pages: waits that pass before the
    page's P V is complete, and waits that nothing can end.  at_end(n): the pages
    whose P V is waited for when n was a tile's last."""
    found, page, known = set(), 0, 0       # known: P V complete whatever the timing
    for length in tiles:
        for k in range(length):
            if k > 0:                      # S of this page was issued behind P V of page - 2
                known = max(known, page - 1)
            waits = [[page - 1]] if k > 0 else []          # where O is rescaled, before P goes out
            if k == length - 1:
                waits.append(at_end(page))
            for i, pages in enumerate(waits):
                most = page + 1 if k == length - 1 and i == len(waits) - 1 else page   # P handed over so far
                low = known
                for w in pages:
                    bar, phase = place(w)
                    for done in range(low, most + 1):
                        count = sum(place(n)[0] == bar for n in range(done))
                        passes = count % 2 != phase % 2
                        if passes and done <= w:
                            found.add("early")
                        if not passes and done == most:
                            found.add("stuck")
                    low = max(low, w + 1)
            page += 1
        known = page                       # the tile's end waited for all of them
    return found


TILES = [t for n in (1, 2, 3, 4) for t in itertools.product((1, 2, 3, 4, 7), repeat=n)]


def test_every_wait_ends_and_none_ends_early(places):
    for tiles in TILES:
        assert not faults(lambda n: places[n], lambda n: [n], tiles), tiles


def test_a_single_barrier_would_not_do():
    """The walk tells: waits for the last two pages in turn on one barrier can
    miss the first of them, and one wait alone can pass early."""
    one = lambda n: (0, n)   # noqa: E731
    assert "stuck" in faults(one, lambda n: [n - 1, n] if n else [n], (3,))
    assert "early" in faults(one, lambda n: [n], (3,))
