"""What the host code of the expert and epilogue calls launches, recorded without
a GPU (tests/host_launch/expert_launches.cpp includes the sources with the launch
replaced): every compiled kernel has a GPU test's shape that reaches it, and the
largest sizes stay inside what a launch holds."""

import os
import re
import shutil
import subprocess

import pytest

from test_gpu_act import FEW as ACT_FEW, GEMMS, GEMMS_LARGE, GRADS
from test_gpu_experts import COMBINES, GATHERS, MANY_ROWS, SORTS
from test_gpu_gemm_experts import FEW, FEW_GATED, ROWS, ROWS_LARGE, SWIGLU, UNALIGNED, VARIANTS, WGRAD, WGRAD_LARGE
from oracle import experts as X

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_launch", "expert_launches.cpp")
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


def calls_of_the_gpu_tests():
    calls = [f"ga {m} {n} {k}" for m, n, k, *_ in GEMMS + GEMMS_LARGE]
    calls += [f"mva {m} {n} {k} {k} {e} 0" for m, n, k in ACT_FEW for e in (0, 1) if k or not e]
    calls += [f"ab {m} {n} {f32} {act} 1" for m, n in GRADS for f32 in (0, 1) for act in range(5)] + ["ab 0 64 0 2 1"]
    calls += [f"sort {t} {k} {e} {align} {size}" for t, k, e in SORTS for align in (1, 32, 256) for size in (4, 8)]
    calls += [f"gat {t} {k} {d} {X.capacity(t * k, e, 32)}" for t, k, e, d in GATHERS]
    calls += [f"gat {t} {k} {d} {X.capacity(t * k, e, align)}" for t, k, e, d, align in MANY_ROWS]
    for t, k, e, d in COMBINES:
        rows = X.capacity(t * k, e, 32)
        calls += [f"com {t} {k} {d} {rows} {z}" for z in (0, 1)] + [f"cob {t} {k} {d} {rows} {dy} {z}" for dy in (0, 1) for z in (0, 1)]

    def padded(sizes, align):
        return sum(-(-s // align) * align for s in sizes)

    calls += [f"ge {len(s)} {padded(s, 32)} {n} {k}" for s, n, k, *_ in ROWS + ROWS_LARGE]
    calls += [f"gw {len(s)} {-(-padded(s, 32) // 256) * 256} {m} {n}" for s, m, n, *_ in WGRAD + WGRAD_LARGE]
    calls += [f"sw {len(s)} {padded(s, 32)} {f} {d}" for s, f, d in SWIGLU]
    calls += [f"mve {len(s)} {sum(s)} {n} {k} {e} 0" for s, n, k in FEW for e in (0, 1)]
    calls += [f"sme {len(s)} {sum(s) + 2} {f} {d} {e} 0" for s, f, d in FEW_GATED for e in (0, 1)]
    for m, n, k in UNALIGNED:
        for e in (0, 1):
            calls += [f"mva {m} {n} {k} {k} {e} 1", f"mve 3 {3 * m} {n} {k} {e} 1", f"sme 3 {3 * m} {n} {k} {e} 1"]
    for m, n, k, off in VARIANTS:
        for e in (0, 1):
            calls.append(f"mva {m} {n} {k} {k} {e} {off}")
            if m <= 16:
                calls += [f"mve 1 {m} {n} {k} {e} {off}", f"sme 1 {m} {n} {k} {e} {off}"]
    return calls


def test_every_kernel_has_a_test_shape(program):
    """The shapes of the GPU tests reach every kernel that is compiled, so that none
    stands untested and none that no call reaches."""
    calls, reached = calls_of_the_gpu_tests(), set()
    for call, (st, made) in zip(calls, launches(program, calls)):
        assert st == 0, call
        reached |= {name.split("::")[-1] for name, _, _ in made}
    symbols = subprocess.run([shutil.which("nm") or "llvm-nm", "-C", program], stdout=subprocess.PIPE, text=True, check=True).stdout
    built = {re.sub(r"\s", "", v) for v in re.findall(r"__device_stub__(\w+_kernel(?:<[^>]*>)?)", symbols)}
    assert len(built) > 80 and reached == built, (sorted(built - reached), sorted(reached - built))


BIG = 1 << 30
_LARGE = [f"sort {BIG} 1 1024 256 4", f"sort {BIG // 8} 8 64 32 8", f"gat {BIG} 1 32 {BIG + (1 << 18)}", f"gat {BIG // 8} 8 {1 << 20} {BIG}",
         f"gat {BIG // 8} 8 160 {BIG}", f"com {BIG // 8} 8 4096 {BIG} 0", f"com {BIG} 1 {BIG} 1 1", f"cob {BIG // 8} 8 32 {BIG} 0 0",
         f"cob 1 {BIG} 64 {BIG} 1 1", f"ab {1 << 40} 32 1 2 1", f"ab 1 {1 << 28} 1 2 1", f"ab {1 << 40} {1 << 28} 0 4 1", f"ge 1024 {BIG} 32 32",
         f"ge 1 {BIG} 65536 256", f"ge 1 5 {BIG} 256", f"gw 1024 {(1 << 24) - 256} 8192 32", f"sw 1024 {BIG} 32 32", f"mve 1024 65536 {1 << 20} 32 0 0",
         f"mve 1 65536 16 4096 0 0", f"sme 1024 65536 17 {(1 << 24) - 32} 0 0", f"mva 64 {1 << 34} 32 32 0 0", f"ga {BIG} 32 32"]


def test_large_launches_stay_below_the_thread_limit(program):
    """A dimension of a launch holds less than 2^32 threads and 65535 rows of workgroups."""
    for call, (st, made) in zip(_LARGE, launches(program, _LARGE)):
        assert st == 0, call
        for name, (x, y, z), threads in made:
            assert 0 < x < 1 << 31 and 0 < y < 1 << 17 and z == 1, (call, name)
            # products: a workgroup a tile, refused past 2^31 - 1 of them
            if "gemm" not in name and "swiglu" not in name:
                assert x * threads < 1 << 32, (call, name)


def test_sorted_rows_have_their_workgroups(program):
    """The products' grids hold every tile that any segments of so many rows make."""
    for experts, rows, n in ((1, 1, 32), (64, 67584, 2048), (8, 9, 300 * 32), (1024, 1024, 32), (3, 255, 288)):
        (st, made), = launches(program, [f"ge {experts} {rows} {n} 256"])
        most = rows // 256 + min(experts + 1, rows)
        assert st == 0 and made[0][1][0] % 8 == 0 and made[0][1][0] >= most * -(-n // 256)
        (st, made), = launches(program, [f"mve {experts} {min(rows, 65536)} {n} 256 0 0"])
        r = min(rows, 65536)
        assert made[0][1][1] == min(experts, r) + r // 16


def test_sizes_whose_small_tiles_pass_a_grid_take_large_ones(program):
    m = n = 1 << 21
    for call in (f"gw 1 256 {m} {n}", f"ga {m} {n} 256", f"ge 1 {m} {n * 128} 256"):
        (st, made), = launches(program, [call])
        assert (st == 0 and "small" not in made[0][0] and 0 < made[0][1][0] < 1 << 31) or (st == 2 and not made), (call, st, made)
    m = n = 1 << 22
    (st, made), = launches(program, [f"gw 1 256 {m} {n}"])
    assert st == 0 and "small" not in made[0][0] and made[0][1][0] == (m // 256) * (n // 256)
