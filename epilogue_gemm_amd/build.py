"""Build the HIP library libgemm_epi.so for gfx950, in-tree.

Every .hip/.cpp file under csrc/ is compiled by hipcc for gfx950 only, in
parallel, then linked into epilogue_gemm_amd/libgemm_epi.so; torch_calls.cpp,
the host-only module that checks torch tensors for binding.py, is compiled by
g++ into _calls.so against the Python and torch headers, where torch is
installed.  build() recompiles everything by default (it is the "does it
build" check); build(incremental=True) (``python -m epilogue_gemm_amd.build --incremental``)
recompiles only the sources whose object is older than the source or any
header it includes (from the compiler's dependency files).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgemm_epi.so")
CALLS_SRC = os.path.join(HERE, "torch_calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # no packed fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


# Per-unit flags.  The row-major-B 16x16x32 tile kernel uses the generic
# machine scheduler: under the default AMDGPU scheduler its accumulators are
# copied between AGPRs and VGPRs around every MFMA (about 400 extra moves
# per two k-steps); the generic one keeps them in place.  Its other kernels
# are built as usual.
UNIT_FLAGS = {
    "gemm_tile16_rowb_f16.hip": ["-mllvm", "-misched=ilpmin"],
    "gemm_tile16_rowb_bf16.hip": ["-mllvm", "-misched=ilpmin"],
}


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _obj(src: str) -> str:
    return os.path.join(BUILD, os.path.basename(src) + ".o")


def _up_to_date(src: str) -> bool:
    """The object exists and is newer than the source and every file its
    dependency file lists."""
    obj, dep = _obj(src), _obj(src) + ".d"
    if not (os.path.exists(obj) and os.path.exists(dep)):
        return False
    t = os.path.getmtime(obj)
    with open(dep) as fh:
        text = fh.read().replace("\\\n", " ")
    files = text.split(":", 1)[1].split() if ":" in text else []
    for f in [src, *files]:
        if not os.path.exists(f) or os.path.getmtime(f) > t:
            return False
    return True


def _compile(src: str) -> str:
    obj = _obj(src)
    extra = UNIT_FLAGS.get(os.path.basename(src), [])
    cmd = [HIPCC, "-x", "hip", *FLAGS, *extra, "-MMD", "-MF", obj + ".d", "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def _build_calls() -> bool:
    """_calls.so; it finds the library beside itself, and torch's libraries
    loaded (binding.py imports torch first).  Not built, and False, where
    torch is not installed: the C library does not need it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return False
    torch = spec.submodule_search_locations[0]
    tmp = CALLS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared", "-isystem", os.path.join(torch, "include"),
           "-I", sysconfig.get_paths()["include"], CALLS_SRC, "-o", tmp, "-L", HERE, "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN", "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALLS_SRC}:\n{r.stderr}")
    os.replace(tmp, CALLS)
    return True


def build(jobs: int | None = None, verbose: bool = False, incremental: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    todo = [s for s in srcs if not (incremental and _up_to_date(s))]
    jobs = jobs or min(max(len(todo), 1), max(1, min(8, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        list(ex.map(_compile, todo))
    if verbose and incremental:
        print(f"compiled {len(todo)} of {len(srcs)} sources: {[os.path.basename(s) for s in todo]}")
    objs = [_obj(s) for s in srcs]
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    calls = CALLS if _build_calls() else f"not {CALLS} (the tensor calls): torch is not installed"
    if verbose:
        print(f"built {LIB} from {len(srcs)} sources, {calls}")
    return LIB


if __name__ == "__main__":
    build(verbose=True, incremental="--incremental" in sys.argv[1:])
    sys.exit(0)
