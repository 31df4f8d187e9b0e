"""The serving step's host side under AddressSanitizer and
UndefinedBehaviorSanitizer: pool.cpp and step.cpp built for the CPU with the HIP
stand-ins of tests/host_check/hip_shim.cpp; tests/host_check/step_driver.cpp runs
random begins between the pool's other operations, predicts their books, checks
the plans and the refusals."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mla_paged_cache_amd", "csrc")
HC = os.path.join(ROOT, "tests", "host_check")
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN = "-fsanitize=address,undefined"
FLAGS = ["-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT}/include", SAN,
         "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not (os.path.exists(CLANG) and os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h")):
        pytest.skip("ROCm clang++ and HIP headers are needed for the host build")
    d = tmp_path_factory.mktemp("host_step")
    srcs = [os.path.join(CSRC, n) for n in ("pool.cpp", "step.cpp", "kvs_mask.cpp")]
    srcs += [os.path.join(HC, n) for n in ("hip_shim.cpp", "step_driver.cpp")]
    objs = [str(d / (os.path.basename(s) + ".o")) for s in srcs]
    procs = [subprocess.Popen([CLANG, "-x", "c++", *FLAGS, "-c", s, "-o", o], stdout=subprocess.PIPE,
                              stderr=subprocess.STDOUT, text=True) for s, o in zip(srcs, objs)]
    for p, s in zip(procs, srcs):
        out, _ = p.communicate()
        assert p.returncode == 0, f"{s}:\n{out}"
    exe = str(d / "step_driver")
    r = subprocess.run([CLANG, SAN, *objs, "-o", exe, "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("kind", ["mla", "gqa"])
@pytest.mark.parametrize("P", [1, 4, 16])
@pytest.mark.parametrize("seed", [0, 1, 2, 3])
def test_random_steps_keep_their_books(driver, kind, P, seed):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=86",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=87")
    r = subprocess.run([driver, kind, str(P), str(seed)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, f"exit {r.returncode}\n{r.stdout}\n{r.stderr[-6000:]}"
    assert "runtime error" not in r.stderr, r.stderr[-6000:]
