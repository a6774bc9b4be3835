"""Row bounds of packed groups, replayed on the host with the library's own rules
(csrc/mm_groups.h): whatever the bounds, the groups that get rows share none, so
the device numbers no more tiles than the host launches for.  A call whose
contraction is split depends on it: one tile per cluster, whose join has no time
limit."""
import ctypes
import os
import random
import subprocess

import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("replay") / "group_replay.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "two_sided_gptq_b200", "csrc"),
                    os.path.join(ROOT, "tests", "cuda", "group_replay.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.replay.restype = lib.launched.restype = ctypes.c_int64
    lib.launched.argtypes = [ctypes.c_int64] * 3

    def replay(offsets, rows, tile, alone=False):
        n = len(offsets) - 1
        has = (ctypes.c_uint8 * n)()
        tiles = lib.replay((ctypes.c_int32 * (n + 1))(*offsets), n, rows, tile, int(alone), has)
        return tiles, list(has)

    return replay, lib.launched


# rows, row bounds, tile of packed rows that the host takes for the call
GOING_BACK = [
    (300, [0, 300, 0, 300], 128),               # two groups of all rows
    (190, [0, 190, 0, 190, 0, 190], 64),        # three of them
    (1000, [0, 1000] * 11, 64),                 # eleven
]


@pytest.mark.parametrize("rows,offsets,tile", GOING_BACK)
def test_bounds_that_go_back_stay_within_the_launch(rules, rows, offsets, tile):
    replay, launched = rules
    bound = launched(rows, len(offsets) - 1, tile)
    # each group's bounds alone would number more tiles than are launched for
    assert replay(offsets, rows, tile, alone=True)[0] > bound
    tiles, has = replay(offsets, rows, tile)
    assert tiles <= bound
    assert has == [1] + [0] * (len(offsets) - 2)


def test_what_counts(rules):
    replay, _ = rules
    for offsets, want in [
        ([0, 5, 5, 9, 10], [1, 1, 1, 1]), ([3, 3, 7, 7], [1, 1, 1]),    # ranges, empty ones among them
        ([0, 50, 40, 100], [1, 0, 0]),                                  # no range; one that begins before row 50
        ([0, 50, 40, 45, 60, 100], [1, 0, 0, 0, 1]),                    # ... until the bounds are past it
        ([50, 40, 60, 70], [0, 1, 1]), ([-1, 10, 20, 30], [0, 1, 1]),   # what is no range takes no rows
        ([0, 10, 101, 20, 30], [1, 0, 0, 1]), ([2 ** 31 - 1, 0, 5, 9], [0, 1, 1]), ([0, 10, -(2 ** 31), 20], [1, 0, 0]),
    ]:
        assert replay(offsets, 100, 64)[1] == want, offsets


@pytest.mark.parametrize("seed", range(4))
def test_any_bounds(rules, seed):
    replay, launched = rules
    rng = random.Random(seed)
    for _ in range(10000):
        experts, rows = rng.choice([1, 2, 3, 5, 21, 40]), rng.choice([1, 7, 64, 190, 300, 1000, 5000])
        near = [0, rows, rows // 2, rows - 1, rows + 1, -1, 2 ** 31 - 1, -(2 ** 31)]
        offsets = [rng.choice(near) if rng.random() < 0.2 else rng.randint(0, rows) for _ in range(experts + 1)]
        if rng.random() < 0.5:
            offsets.sort()
        for tile in (64, 128, 256):
            tiles, has = replay(offsets, rows, tile)
            assert tiles <= launched(rows, experts, tile), (rows, offsets, tile)
        taken = [(a, b) for a, b, h in zip(offsets, offsets[1:], has) if h]
        assert all(0 <= a <= b <= rows for a, b in taken)
        assert all(b <= c for (_, b), (c, _) in zip(taken, taken[1:])), offsets
        if offsets == sorted(offsets) and offsets[0] >= 0 and offsets[-1] <= rows:
            assert all(has)
