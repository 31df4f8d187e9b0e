"""The serving step's host side at its limits, on the CPU under the sanitizers of
test_host_step.py: tests/host_check/step_limits_driver.cpp, one check a run."""

import os
import subprocess

import pytest

from test_host_step import CLANG, CSRC, FLAGS, HC, SAN

CHECKS = ["eager_calls_beside_a_graph", "growth", "tables_behind_an_eviction", "queries_in_place", "scales",
          "shares_of_long_tiles"]


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not (os.path.exists(CLANG) and os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h")):
        pytest.skip("ROCm clang++ and HIP headers are needed for the host build")
    d = tmp_path_factory.mktemp("host_step_limits")
    srcs = [os.path.join(CSRC, n) for n in ("pool.cpp", "step.cpp", "kvs_mask.cpp")]
    srcs += [os.path.join(HC, n) for n in ("hip_shim.cpp", "step_limits_driver.cpp")]
    objs = [str(d / (os.path.basename(s) + ".o")) for s in srcs]
    procs = [subprocess.Popen([CLANG, "-x", "c++", *FLAGS, "-Wno-unused-function", "-c", s, "-o", o],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for s, o in zip(srcs, objs)]
    for p, s in zip(procs, srcs):
        out, _ = p.communicate()
        assert p.returncode == 0, f"{s}:\n{out}"
    exe = str(d / "step_limits_driver")
    r = subprocess.run([CLANG, SAN, *objs, "-o", exe, "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("check", CHECKS)
def test_limit(driver, check):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=86",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=87")
    r = subprocess.run([driver, check], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, f"exit {r.returncode}\n{r.stdout}\n{r.stderr[-6000:]}"
    assert "runtime error" not in r.stderr, r.stderr[-6000:]
