"""The host code of the expert and epilogue calls under AddressSanitizer and
UndefinedBehaviorSanitizer, with the launches replaced by a record (host code
only, on the CPU): the calls of the GPU tests, the largest sizes, and arguments
far outside what the calls take."""

import itertools
import os
import subprocess

import pytest

from test_expert_launch_rules import _LARGE, HIPCC, SRC, calls_of_the_gpu_tests

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")

MAX, MIN = (1 << 63) - 1, -(1 << 63)
EXTREME = (MIN, -1, 0, 1, 33, 256, 1 << 24, 1 << 31, 1 << 40, MAX - 31, MAX)
OPS = {"ga": 3, "mva": 4, "ab": 2, "sort": 4, "gat": 4, "com": 4, "cob": 4, "ge": 4, "gw": 4, "sw": 4, "mve": 4, "sme": 4}
REST = {"mva": "0 0", "ab": "1 2 1", "sort": "4", "com": "0", "cob": "1 0", "mve": "0 0", "sme": "0 0"}


def test_host_code_is_clean(tmp_path):
    exe = str(tmp_path / "checks")
    cmd = [HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g", "-std=c++17", "-x", "hip", SRC, "-o", exe, "-rdynamic",
           "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer",
           "-Wl,--unresolved-symbols=ignore-all"]
    b = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=600)
    assert b.returncode == 0, b.stdout.decode()[-4000:]
    calls = calls_of_the_gpu_tests() + _LARGE
    for op, n in OPS.items():
        for base in itertools.product((1, 64), repeat=n):   # one argument extreme, then two
            for i, j in itertools.combinations_with_replacement(range(n), 2):
                for x, y in ((x, y) for x in EXTREME for y in (EXTREME if j > i else (0,))):
                    v = list(base)
                    v[i], v[j] = x, y if j > i else x
                    calls.append(f"{op} {' '.join(map(str, v))} {REST.get(op, '')}")
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], input="\n".join(calls) + "\n", stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, \
        (calls[len(r.stdout.splitlines())] if r.returncode else "", r.stderr[-3000:])
    status = [int(line.split()[0]) for line in r.stdout.splitlines()]
    assert len(status) == len(calls) and set(status) <= {0, 1, 2, 3}
