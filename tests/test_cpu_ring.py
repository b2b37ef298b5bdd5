"""The ring of the row-wise forward, replayed on the host: whether the producer
gets every slot back, for whole and short groups of rows and both directions.
The rule for the rows that a short group lacks is read from the kernel."""
import os
import re

import pytest

import mxfp8_quantization_gb300 as rn

CSRC = os.path.join(os.path.dirname(os.path.abspath(rn.__file__)), "csrc")


def missing_rows_arrive():
    """Whether the kernel's branch for a row past the end gives the slot back, in its turn: after the wait for the
    slot's previous use."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "rn_fwd.cu")).read())
    k = text[text.index("rn_fwd_kernel(const FwdParams p)"):]
    at = re.search(r"if \(r >= p\.N\)\s*(\{[^}]*\}|continue;)", k)
    turn = k.index("mbar_wait(smem_u32(&empty[s]), pos.phase ^ 1u, &g_err_fwd, kErrStatsWait)")
    return "mbar_arrive(smem_u32(&empty[s]))" in at.group(1) and turn < at.start()


def replay(N, rps, Q, grid, reverse):
    """Every CTA's producer and groups of warps, as far as they get; the slots that never come back."""
    arrive = missing_rows_arrive()
    groups = -(-N // rps)
    stuck = []
    for b in range(min(grid, groups)):
        count = (groups - b + grid - 1) // grid
        first = b + (count - 1) * grid if reverse else b
        given = [0] * count          # arrivals for each use of a slot
        for kg in range(count):
            start = (first + kg * (-grid if reverse else grid)) * rps
            for j in range(rps):
                given[kg] += start + j < N or arrive
        for i in range(Q, count):    # the producer waits for use i - Q of the slot
            if given[i - Q] < rps:
                stuck.append((b, i))
    return stuck


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("N,rps,Q", [(17594, 4, 21), (65537, 8, 27), (20001, 4, 27), (16385, 2, 27), (16384, 2, 27)])
def test_every_slot_comes_back(N, rps, Q, reverse):
    assert not replay(N, rps, Q, 152, reverse)
