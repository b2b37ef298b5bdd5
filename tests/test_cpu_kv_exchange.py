"""The statistics that the odd pages' warps of the attention's tiles hand to the even pages' warps, replayed on the
host: whether every one is read before its place is written again, by what the warps wait for and not by how fast they
are.  The places and whose turn it is are read from the kernel."""
import itertools
import os
import re

import pytest

import mxfp8_quantization_gb300 as rn

CSRC = os.path.join(os.path.dirname(os.path.abspath(rn.__file__)), "csrc")


def places():
    """How many places the segments take in turn."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "rn_kv_tile.cu")).read())
    k = text[text.index("rn_kv_tile_kernel(const KvAttnParams p"):]
    n = re.search(r"__shared__ Stats other\[(\d+)\]\[128\]", k)
    if n is None:
        return 1
    # one index for the write and the read, changed once a segment, behind the read
    write, bar = k.index("other[turn][in_tile] = Stats"), k.index("bar.sync 1, 256;")
    read, change = k.index("= other[turn][in_tile];"), k.index("turn ^= 1;")
    assert write < bar < read < change and k.count("turn ^= 1;") == 1 and k.count("other[") == 3
    return int(n.group(1))


def order(segments):
    """What comes before what: {event: the events right before it}.  A segment is (pages, both): `both` where the tile
    has more than 128 rows, whose two halves take every page; else the pages go to the two groups in turn."""
    before, last = {}, {"even": None, "odd": None, "products": None}

    def step(who, event, *others):
        before.setdefault(event, set()).update(x for x in (last[who], *others) if x is not None)
        last[who] = event

    for k, (pages, both) in enumerate(segments):
        for who in ("even", "odd"):
            step(who, ("queries", who, k))
        step("products", ("products", k), ("queries", "even", k), ("queries", "odd", k))
        step("even", ("output", "even", k), ("products", k))
        step("odd", ("output", "odd", k), *[("products", k)] * (both or pages > 1))
        if not both:
            step("odd", ("write", k))
            for who in ("even", "odd"):
                step(who, ("met", who, k))
            for event in (("met", "even", k), ("met", "odd", k)):
                before[event] |= {("write", k), ("output", "even", k)}
            step("even", ("read", k))
    return before


def comes_before(before, a, b):
    todo, seen = [b], set()
    while todo:
        x = todo.pop()
        if x == a:
            return True
        if x not in seen:
            seen.add(x)
            todo.extend(before.get(x, ()))
    return False


def unordered(segments, n):
    before = order(segments)
    split = [k for k, (_, both) in enumerate(segments) if not both]
    bad = [(k, "read") for k in split if not comes_before(before, ("write", k), ("read", k))]
    return bad + [(a, b) for i, a in enumerate(split) for b in split[i + n:i + n + 1]
                  if not comes_before(before, ("read", a), ("write", b))]


def test_one_place_would_not_do():
    assert unordered([(2, False), (1, False)], 1) == [(0, 1)]
    assert unordered([(2, False), (2, False), (3, True), (1, False)], 1) == []


@pytest.mark.parametrize("length", range(1, 6))
def test_every_place_is_read_before_it_is_written_again(length):
    kinds = [(1, False), (2, False), (3, False), (1, True), (2, True)]
    for segments in itertools.product(kinds, repeat=length):
        assert unordered(segments, places()) == [], segments
