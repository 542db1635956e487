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


# t at and around 2^32 threads for each number of rows a workgroup holds, and the largest that the call takes
@pytest.mark.parametrize("d", [32, 128, 160, 2048, 2080, 8192, 16384, 32768])
@pytest.mark.parametrize("t", [1, 8192, (1 << 22) - 1, 1 << 22, (1 << 23) + 5, (1 << 24) - 1, 1 << 24, (1 << 26) + 3, 1 << 28,
                               (1 << 28) + 17, (1 << 31) - 1])
def test_norm_launches_stay_below_the_thread_limit(program, t, d):
    """A dimension of a launch holds less than 2^32 threads; every row has its workgroup."""
    for op in ("norm", "bwd"):
        for st, made in launches(program, [f"{op} {t} {d} {f32} {extra}" for f32 in (0, 1) for extra in (0, 1)]):
            assert st == 0
            for name, (x, y, z), threads in made:
                assert x * threads < 1 << 32 and y < 1 << 16 and z == 1, name
            name, (x, y, z), _ = made[0]
            lanes = int(re.search(r"<(\d+),", name)[1])
            rows = max(256 // lanes, 1)
            if op == "norm":
                assert x * y * rows >= t and x * (y - 1) * rows < t
            else:
                assert x <= 512 and y == 1
