"""Which tiles the products over sorted rows take: the faster ones of measured shapes
(operands from memory, a difference of 5% and more)."""

import os

import pytest

from test_expert_launch_rules import HIPCC, launches, program  # noqa: F401 (a fixture)

# (experts, rows with padding, n, k), us in large and in small tiles
SHAPES = [((64, 2560, 2048, 2048), 48.4, 41.7), ((64, 4096, 2048, 2048), 55.5, 49.7), ((64, 10240, 2048, 2048), 66.0, 83.7),
          ((8, 768, 14336, 4096), 80.0, 111.4), ((8, 512, 14336, 4096), 70.6, 84.9),
          ((8, 64, 14336, 4096), 63.8, 57.2), ((8, 512, 28672, 4096), 136.3, 158.1), ((8, 64, 28672, 4096), 129.4, 110.3),
          ((16, 768, 4096, 4096), 60.8, 49.7), ((16, 1024, 4096, 4096), 44.6, 56.9), ((32, 1280, 4096, 4096), 93.4, 78.8),
          ((8, 512, 4096, 14336), 93.9, 87.8), ((8, 1024, 4096, 4096), 38.3, 43.9), ((8, 64, 4096, 14336), 89.4, 58.3),
          ((128, 4608, 1024, 1024), 26.9, 25.3),
          ((128, 6144, 2048, 768), 50.9, 45.0), ((48, 2560, 512, 512), 9.9, 6.5), ((8, 2304, 1024, 1024), 14.7, 9.7)]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("shape,large,small", SHAPES)
def test_the_faster_tiles(program, shape, large, small):  # noqa: F811
    (st, ((name, _, _),)), = launches(program, ["ge " + " ".join(map(str, shape))])
    assert st == 0 and ("small" in name) == (small < large)
