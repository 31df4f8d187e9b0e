"""Build the gfx950 library libleyline.so in-tree with hipcc.

The library holds the HIP kernels (csrc/kernels.hip for MLA pools,
csrc/kernels_gqa.hip for GQA / MHA pools, csrc/kernels_kvs.hip for the
KV-streams trainer mask, csrc/kernels_rows.hip for the per-row-angle
rotation, csrc/kernels_alloc.hip for the eviction's device-side page
allocator, csrc/kernels_step.hip and csrc/kernels_attend.hip for the serving
step, csrc/kernels_weigh.hip and csrc/kernels_keep.hip for eviction by
attention weight, csrc/kernels_train.hip and csrc/kernels_train_back.hip for
the trainer's attention, helpers in csrc/device_common.h,
csrc/matrix_common.h and csrc/train_common.h) and the C++ host side and C ABI
(csrc/pool.cpp, csrc/step.cpp, csrc/weight.cpp, csrc/kvs_mask.cpp,
csrc/train.cpp).  Flags:
  * --offload-arch=gfx950 only (MI355X);
  * -ffp-contract=off so the delta-rotation keeps its separately rounded
    float32 products (the kernels also say so with a pragma);
  * -target-feature -packed-fp32-ops keeps the compiler away from packed fp32
    instructions.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libleyline.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)

SOURCES = [os.path.join(CSRC, n) for n in ("kernels.hip", "kernels_gqa.hip", "kernels_kvs.hip", "kernels_rows.hip",
                                           "kernels_alloc.hip", "kernels_step.hip", "kernels_attend.hip",
                                           "kernels_weigh.hip", "kernels_keep.hip", "kernels_train.hip",
                                           "kernels_train_back.hip", "pool.cpp", "step.cpp", "weight.cpp",
                                           "kvs_mask.cpp", "train.cpp")]

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Winfinite-recursion",
    # host code: the hardware popcount (the free-page bitmap is merged and
    # counted word by word; without it every popcount is a dozen ALU ops)
    "-Xarch_host", "-mpopcnt",
]

# Matrix accumulators in ordinary registers: the attention scales and stores them, and
# moving each to and from the accumulation file costs more than the products (the
# compiler's own choice otherwise).  Not where the sums alone fill that file.
VGPR_SUMS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
OWN_SUMS = ("kernels_train_back.hip",)


def flags(source: str) -> list:
    return FLAGS + ([] if os.path.basename(source) in OWN_SUMS else VGPR_SUMS)


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the gfx950 library cannot be built")


def build(verbose: bool = False) -> str:
    """Compile libleyline.so next to this file, its sources side by side; returns
    its path."""
    noise = ("not a recognized feature for this target", "ignoring feature")

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        err = "\n".join(l for l in (res.stderr or "").splitlines() if not any(w in l for w in noise))
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
        return err

    tmp = LIB_PATH + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        compiles = [[hipcc(), *flags(s), "-I", INCLUDE, "-c", s, "-o", o] for s, o in zip(SOURCES, objects)]
        link = [hipcc(), "--offload-arch=gfx950", "-shared", "-Wl,--no-undefined", *objects, "-o", tmp]
        if verbose:
            print(" ".join(compiles[0]), flush=True)
        with concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            errs = list(pool.map(run, compiles))
        errs.append(run(link))
    err = "\n".join(e for e in errs if e.strip())
    if verbose and err:
        print(err)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
