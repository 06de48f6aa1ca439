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


def faults(place, lag, at_end, tiles):
    """What can go wrong over tiles of so many pages: waits that pass before the
    page's P V is complete, and waits that nothing can end.  lag: each page waits
    for the page so many before it (None: it does not); at_end(n): the pages that
    are waited for one after the other when n was a tile's last.  Nothing but a wait
    tells of P V."""
    found, page = set(), 0
    low = 0                                # P V known to be complete
    for length in tiles:
        for k in range(length):
            # (for which page, P handed over by then, whether it is made every time)
            waits = [(page - lag, page, True)] if lag and page >= lag else []
            if k > 0:
                waits.append((page - 1, page, False))      # where O is rescaled
            if k == length - 1:
                waits += [(n, page + 1, True) for n in at_end(page)]
            for n, most, always in waits:
                bar, phase = place(n)
                for done in range(low, most + 1):
                    passes = sum(place(m)[0] == bar for m in range(done)) % 2 != phase % 2
                    if passes and done <= n:
                        found.add("early")
                    if not passes and done == most:
                        found.add("stuck")
                if always:
                    low = max(low, n + 1)
            page += 1
    return found


TILES = [t for n in (1, 2, 3, 4) for t in itertools.product((1, 2, 3, 4, 7), repeat=n)]


def test_every_wait_ends_and_none_ends_early(places):
    for tiles in TILES:
        assert not faults(lambda n: places[n], 2, lambda n: [n], tiles), tiles


def test_other_rules_would_not_do(places):
    """The walk tells: on one barrier, waits for the last two pages in turn can
    miss the first of them; without a wait for every page, one can pass early on
    a phase that nobody saw."""
    one = lambda n: (0, n)   # noqa: E731
    assert "stuck" in faults(one, None, lambda n: [n - 1, n] if n else [n], (3,))
    assert "early" in faults(one, None, lambda n: [n], (3,))
    assert "early" in faults(lambda n: places[n], None, lambda n: [n], (4,))
