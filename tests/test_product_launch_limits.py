"""A dimension of a launch holds less than 2^32 threads: products of more tiles than
that take a second one, and every tile has its workgroup."""

import os

import pytest

from test_expert_launch_rules import HIPCC, _LARGE, launches, program  # noqa: F401 (a fixture)

# (call, tiles of 256 x 256, of 256 x 128 for the gated producer, of 64 x 64)
BIG = 1 << 30
CASES = [("ge 1024 1024 1048576 32", 1028 * 4096, 1040 * 16384), ("ge 1024 1024 4194304 32", 1028 * 16384, 1040 * 65536),
         ("ge 1024 98304 1048576 32", 1409 * 4096, 2561 * 16384), (f"ge 1 {BIG} 65536 256", (4194304 + 2) * 256, 0),
         ("ge 1 1 1073741824 32", 1 << 22, 1 << 24), ("ga 1 2147483648 32", 1 << 23, 0), ("ga 2147483905 32 32", (1 << 23) + 2, 0),
         ("ga 257 1073742112 32", 2 * (4194304 + 2), 0), ("ga 1 1073741824 32", 1 << 22, 0), ("ga 1 1073742080 32", (1 << 22) + 1, 0),
         ("gw 1024 256 32 1048576", 1 << 22, 0), ("gw 1024 256 32 1048832", (1 << 22) + 1024, 0), ("gw 1 256 4194304 4194304", 1 << 28, 0),
         ("sw 1024 1024 524288 32", 1028 * 4096, 0), ("sw 1024 32768 4194304 32", 1153 * 32768, 0)]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("call,large,small", CASES)
def test_every_tile_has_its_workgroup(program, call, large, small):  # noqa: F811
    (st, ((name, (x, y, z), threads),)), = launches(program, [call])
    tiles = small if "small" in name else large
    assert st == 0 and z == 1 and x * threads < 1 << 32 and y < 1 << 16
    assert tiles <= x * y < tiles + 8 * y and (y == 1 or x % 8 == 0)


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_no_launch_passes_the_thread_limit(program):  # noqa: F811
    for call, (st, made) in zip(_LARGE, launches(program, _LARGE)):
        assert st == 0 and all(x * threads < 1 << 32 and y < 1 << 16 for _, (x, y, _z), threads in made), call


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_more_tiles_than_any_launch_are_refused(program):  # noqa: F811
    for call in ("ga 1073741824 131072 256", f"ge 1 {BIG} 131072 256", "gw 1024 256 1048576 131072", f"sw 1 {BIG} 131072 256"):
        assert launches(program, [call]) == [(2, [])], call
