"""The cut of draft trees by rows (csrc/decode_tree_tc.cu), replayed on the host: which parts of groups a CTA takes, one after
the other.  The shapes of test_gpu_tree_cut are chosen by what their cut does; this file says that they still do it."""
import os
import re

import pytest

from long_context_sparse_dsa_gb300 import build as dsa_build


def _constants():
    with open(os.path.join(dsa_build.CSRC, "decode_tree_tc.cu")) as f:
        text = f.read()
    find = lambda p: int(re.search(p, text).group(1))  # noqa: E731
    return (find(r"constexpr int kTcSms = (\d+);"), find(r"constexpr int kGroupRows = (\d+);"), find(r"constexpr int kTileKeys = (\d+);"),
            find(r"a\.min_tiles = (\d+);"))


def segments(lens, nodes, Hq):
    """Of every CTA its segments in order: (query rows of the group, first key tile, end, key tiles of the group)."""
    ctas, group, tile, least = _constants()
    parts = []   # (query rows, tiles) of the groups, in order
    for n, m in zip(lens, nodes):
        for g in range(-(-m * Hq // group)):
            parts.append((min(group, m * Hq - g * group), -(-n // tile) + 1))
    total = sum(t for _, t in parts)
    per = max(-(-total // ctas), least)
    out, at = [[] for _ in range(ctas)], 0
    for rows, tiles in parts:
        t = 0
        while t < tiles:
            end = min(tiles, t + per - (at + t) % per)
            out[(at + t) // per].append((rows, t, end, tiles))
            t = end
        at += tiles
    return out


def hand_overs(lens, nodes, Hq):
    """Places where, in one CTA, the second accumulator has units in a group of up to 128 query rows, and none in the next
    segment, whose last tile is not the group's: nothing but the barrier behind the sums keeps its warps from writing again."""
    n = 0
    for cta in segments(lens, nodes, Hq):
        for (rows, a, b, _), (rows2, a2, b2, tiles2) in zip(cta, cta[1:]):
            n += rows <= 128 and b - a >= 2 and rows2 <= 128 and b2 - a2 == 1 and b2 < tiles2
    return n


def _ragged(batch, most, seed):
    x = [1 + (b * 7919 + seed) % most for b in range(batch)]
    x[0] = most
    return x


# (lens, nodes, query heads, d)
SHAPES = {
    "64 of 8 over 2048": ([2048] * 64, [8] * 64, 16, 128),
    "64 of 8 over 4000": ([4000] * 64, [8] * 64, 16, 128),
    "64 of 8 over 4000, d 64": ([4000] * 64, [8] * 64, 16, 64),
    "128 of 4 over 4096": ([4096] * 128, [4] * 128, 32, 128),
    "24 of 3 over 2000": ([2000] * 24, [3] * 24, 16, 128),
    "24 of 3 over 2000, d 64": ([2000] * 24, [3] * 24, 16, 64),
    "ragged 90": (_ragged(90, 3500, 61), [1 + b % 8 for b in range(90)], 16, 128),
    "ragged 40": (_ragged(40, 9000, 17), [1 + b * 5 % 8 for b in range(40)], 16, 64),
    "ragged 200": (_ragged(200, 2000, 5), [b % 5 for b in range(200)], 32, 128),
}


def test_the_cut_covers_every_tile_once():
    for lens, nodes, Hq, _ in SHAPES.values():
        whole = [(min(256, m * Hq - g), -(-n // 128) + 1) for n, m in zip(lens, nodes) for g in range(0, m * Hq, 256)]
        flat = [x for cta in segments(lens, nodes, Hq) for x in cta]
        got, t = [], 0
        for rows, a, b, tiles in flat:
            assert a == t and b > a
            t = 0 if b == tiles else b
            if b == tiles:
                got.append((rows, tiles))
        assert got == whole


@pytest.mark.parametrize("name", SHAPES)
def test_the_shapes_hand_over_to_a_single_tile(name):
    lens, nodes, Hq, _ = SHAPES[name]
    assert hand_overs(lens, nodes, Hq) > 0


def test_one_long_row_does_not():
    assert hand_overs([131069], [16], 16) == 0


def test_the_sums_are_handed_over_between_two_barriers():
    """Each half of the second accumulator's sums is written, met by a barrier, read, and met by another, whichever half it is: on
    the GPU only the timing would show a missing one."""
    with open(os.path.join(dsa_build.CSRC, "decode_tree_tc.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    block = text[text.index("float* box = reinterpret_cast<float*>(smem + C::TILE)"):]
    block = block[:block.index("if (live && (both || g == 0))")]
    write, meet, read, leave = (block.index(x) for x in ("box[(32 * c + e) * 128 + r] = o[e]", "tc_bar(1, 256)", "f1 * box[(32 * c",
                                                         "m = fmaxf(m, box_ml[r].x)"))
    assert write < meet < read < leave < block.rindex("tc_bar(1, 256)")
    assert not re.search(r"(if|else)[^;{}]*tc_bar\(", block)
