"""What the host code of the norm, dropout and few-row product calls launches,
recorded without a GPU (tests/host_launch/launches.cpp includes the sources
with the launch replaced)."""

import os
import re
import shutil
import subprocess

import pytest

from test_gpu_matvec_variants import KINDS, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_launch", "launches.cpp")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("launches") / "launches")
    # host code alone: the device image that it refers to is left out
    cmd = [HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-x", "hip", SRC, "-o", exe, "-rdynamic",
           "-Wl,--unresolved-symbols=ignore-all"]
    b = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    assert b.returncode == 0, b.stdout.decode()[-4000:]
    return exe


def launches(program, calls):
    """(status, [(kernel, (grid x, y, z), threads)]) of each call."""
    r = subprocess.run([program], input="\n".join(calls) + "\n", stdout=subprocess.PIPE, text=True, timeout=120)
    assert r.returncode == 0
    out = []
    for line in r.stdout.splitlines():
        st, *w = line.split()
        out.append((int(st), [(w[i], tuple(map(int, w[i + 1:i + 4])), int(w[i + 4])) for i in range(0, len(w), 5)]))
    assert len(out) == len(calls)
    return out


def test_every_product_variant_has_a_test_shape(program):
    """The shapes of test_gpu_matvec_variants reach all variants that are
    compiled, so that none stands untested and none that no call reaches."""
    calls = [f"mv {m} {n} {k} {k} {kind == 'e4m3':d} {off}" for m, n, k, off in SHAPES for kind in KINDS]
    calls += [f"sw {m} {n} {k} {k} {kind == 'e4m3':d} {off}" for m, n, k, off in SHAPES for kind in KINDS]
    calls += [f"nv {m} {n} {k} {k} {off}" for m, n, k, off in SHAPES]
    reached = set()
    for call, (st, made) in zip(calls, launches(program, calls)):
        assert st == 0 and len(made) == 1, call
        name, grid, threads = made[0]
        assert 1 <= grid[0] <= 256 and grid[1:] == (1, 1) and threads in (512, 1024), call
        reached.add(name)
    symbols = subprocess.run([shutil.which("nm") or "llvm-nm", "-C", program], stdout=subprocess.PIPE, text=True, check=True).stdout
    built = {re.sub(r"\s", "", v) for v in re.findall(r"__device_stub__(matvec_kernel<[^>]*>)", symbols)}
    compiled = {name.split("::")[-1] for name in reached}
    assert len(built) > 70 and compiled == built, sorted(built - compiled)
