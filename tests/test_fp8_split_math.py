"""The balanced split of the 8-bit decode on the host: the arithmetic is the
kernels' own header, compiled here; the work list around it is restated.

A unit is (sequence, group of KV heads).  Its tiles start at the unit's position
+ UNIT_COST, a tile's cost apart; group c of C takes the tiles that start in
[c W / C, (c + 1) W / C).  The reduce reads one partial slot of a unit for each group
from that of the unit's first tile to that of its last, so every one of them must
have a tile of the unit: a slot that nobody wrote holds whatever the workspace did."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "fp8_split.h"
using namespace attn;
extern "C" {
int unit_cost() { return kFp8UnitCost; }
int most_tile_cost() { return kFp8MostTileCost; }
int cost_of_columns(int n) { return fp8_cost_of_columns(n); }
int split_groups(int g, int T, int W, int d) { return fp8_split_groups(g, T, W, d); }
int position(int c, int W, int C) { return first_position(c, W, C); }
int group_of(int y, int W, int C) { return group_of_position(y, W, C); }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I",
                    os.path.join(ROOT, "split_flash_decoding_gb300", "csrc"), str(d / "shim.cpp"),
                    "-o", str(d / "shim.so")], check=True)
    return ctypes.CDLL(str(d / "shim.so"))


def unwritten(split, groups, heads, tiles, costs):
    """Slots that the reduce reads and no group wrote; also that tiles are all dealt
    out.  tiles, costs: of each sequence; heads: groups of KV heads."""
    opening = split.unit_cost()
    units, at = [], 0
    for n, cost in zip(tiles, costs):
        for _ in range(heads):
            first = at + opening
            units.append((first, first + (n - 1) * cost, n, cost))
            at += opening + n * cost
    T, W = heads * sum(tiles), at
    C = split.split_groups(groups, T, W, max(costs))
    assert 1 <= C <= min(groups, T)
    starts = [split.position(c, W, C) for c in range(C)] + [W]
    assert starts[0] == 0 and all(a < b for a, b in zip(starts, starts[1:]))
    missing = 0
    for first, last, n, cost in units:
        c0, c1 = split.group_of(first, W, C), split.group_of(last, W, C)
        assert starts[c0] <= first < starts[c0 + 1] and starts[c1] <= last < starts[c1 + 1]
        dealt = 0
        for c in range(c0, c1 + 1):
            lo, hi = max(starts[c], first), min(starts[c + 1] - 1, last)
            here = (hi - first) // cost - (lo - first + cost - 1) // cost + 1 if hi >= lo else 0
            missing += here <= 0
            dealt += max(here, 0)
        assert dealt == n
    return missing


def test_costs(split):
    assert [split.cost_of_columns(n) for n in (0, 1, 4, 5, 8, 9, 12, 13, 16, 40)] == \
        [8, 8, 8, 9, 9, 10, 10, 11, 11, 11]
    assert split.most_tile_cost() == split.cost_of_columns(16)


@pytest.mark.parametrize("hkv,rows,keys", [
    (1, [1, 4], [32000, 6900]), (8, [1, 4], [2944, 768]), (1, [4, 1], [2560, 35840]),
    (1, [1, 4], [30000, 3000]), (2, [4, 1, 1, 1], [4096] * 4)])
def test_unequal_rows_leave_no_slot_unwritten(split, hkv, rows, keys):
    side = min(hkv, 8)
    tiles = [-(-k // 128) for k in keys]
    costs = [split.cost_of_columns(4 * r) for r in rows]
    assert unwritten(split, 304 // side, hkv // side, tiles, costs) == 0


def test_random_mixes_leave_no_slot_unwritten(split):
    rng = random.Random(5)
    for _ in range(4000):
        group = rng.choice([1, 2, 3, 4, 5, 8])
        groups, heads = rng.choice([1, 7, 38, 76, 152, 304]), rng.choice([1, 1, 2, 3])
        batch = rng.randint(1, 8)
        # around as many tiles as groups, where ranges are shortest
        most = max(1, int(groups * rng.uniform(0.3, 4.0)) // (batch * heads))
        tiles = [rng.randint(1, most) if rng.random() < 0.8 else rng.randint(1, 4 * most)
                 for _ in range(batch)]
        costs = [split.cost_of_columns(rng.randint(1, 16 // group) * group) for _ in range(batch)]
        assert unwritten(split, groups, heads, tiles, costs) == 0, (groups, heads, tiles, costs)


def test_equal_rows_use_every_group_that_has_a_tile(split):
    for cost in (8, 9, 10, 11):
        for T in (1, 5, 100, 304, 1000):
            W = T * cost + split.unit_cost()
            assert split.split_groups(304, T, W, cost) == min(304, T)
