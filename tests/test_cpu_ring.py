"""The ring of the row-wise forward, replayed on the host: whether the producer
gets every slot back, for whole and short groups of rows and both directions.
The rule for the rows that a short group lacks is read from the kernel."""
import os
import re

import pytest

import mxfp8_quantization_gb300 as rn

CSRC = os.path.join(os.path.dirname(os.path.abspath(rn.__file__)), "csrc")


def missing_rows_arrive():
    """For rows past the end: whether the kernel's branch gives their part of the slot back when the rows are walked
    backwards (in the passes that do so); it may not where the slot could still be in its previous use."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "rn_fwd.cu")).read())
    k = text[text.index("rn_fwd_kernel(const FwdParams p)"):]
    start = at = k.index("{", k.index("if (r >= p.N)")) if "if (r >= p.N) {" in k else None
    if start is None:
        return False
    depth = 1
    while depth:
        at += 1
        depth += (k[at] == "{") - (k[at] == "}")
    branch = k[start:at]
    return re.search(r"if \(PASS2 && p\.reverse\) \{\s*__syncwarp\(\);\s*if \(lane == 0\) "
                     r"mbar_arrive\(smem_u32\(&empty\[pos\.slot\]\)\);\s*\}\s*continue;", branch) is not None


def test_only_the_second_passes_walk_backwards():
    api = open(os.path.join(CSRC, "rn_api.cu")).read()
    launches = re.findall(r"q\.reverse = 1;(.{0,900}?)launch_fwd(?:_res)?\([^;]*?(kQ\w+)", api, flags=re.S)
    assert [q for _, q in launches] and {q for _, q in launches} <= {"kQNvfp4", "kQCurQuant"}


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
                given[kg] += start + j < N or (arrive and reverse)
            if start + rps > N:
                assert kg == (0 if reverse else count - 1)       # no previous use, or none to come
        for i in range(Q, count):    # the producer waits for use i - Q of the slot
            if given[i - Q] < rps:
                stuck.append((b, i))
    return stuck


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("N,rps,Q", [(17594, 4, 21), (65537, 8, 27), (20001, 4, 27), (16385, 2, 27), (16384, 2, 27)])
def test_every_slot_comes_back(N, rps, Q, reverse):
    assert not replay(N, rps, Q, 152, reverse)
