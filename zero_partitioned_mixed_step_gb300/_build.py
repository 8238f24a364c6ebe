"""Build libzerostep.so (the step), libzerostep_ops.so (the operators around it)
and libzerostep_layer.so (what lies between a layer's products) in-tree with nvcc
for sm_103a."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libzerostep.so")
OPS = os.path.join(CSRC, "ops")
OPS_LIB = os.path.join(BUILD, "libzerostep_ops.so")
LAYER = os.path.join(CSRC, "layer")
LAYER_LIB = os.path.join(BUILD, "libzerostep_layer.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    """The CUDA compiler: on PATH, else under CUDA_HOME or /usr/local/cuda."""
    found = shutil.which("nvcc")
    if found:
        return found
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found (install the CUDA toolkit or set CUDA_HOME)")
    return path
# -fmad=false keeps device arithmetic uncontracted; -ffp-contract=off does the
# same for the host code (the host rounds configuration-only scalars).
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-fmad=false", "-Xcompiler", "-ffp-contract=off",
              "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-Xcompiler", "-Wall", "-I", INCLUDE, *ARCH]
# The operators' arithmetic has no oracle to match bit for bit: contraction is allowed.
OPS_NVCC_FLAGS = [f for f in NVCC_FLAGS if f != "-fmad=false"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _inputs():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "zerostep.h"), __file__]


def _ops_sources():
    return sorted(glob.glob(os.path.join(OPS, "*.cu")))


def _ops_inputs():
    return _ops_sources() + glob.glob(os.path.join(OPS, "*.cuh")) + [
        os.path.join(INCLUDE, "zerostep.h"), os.path.join(INCLUDE, "zerostep_ops.h"), __file__]


def _layer_sources():
    return sorted(glob.glob(os.path.join(LAYER, "*.cu")))


def _layer_inputs():
    return _layer_sources() + glob.glob(os.path.join(LAYER, "*.cuh")) + [
        os.path.join(OPS, "ops.cuh"), os.path.join(INCLUDE, "zerostep.h"), os.path.join(INCLUDE, "zerostep_ops.h"),
        os.path.join(INCLUDE, "zerostep_layer.h"), __file__]


def _older(lib: str, inputs) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in inputs)


def stale() -> bool:
    return (_older(LIB, _inputs()) or _older(OPS_LIB, _ops_inputs())
            or _older(LAYER_LIB, _layer_inputs()))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit of the libraries in parallel and link
    them.  Returns the step library's path."""
    todo = [(lib, sources(), flags)
            for lib, sources, inputs, flags in ((LIB, _sources, _inputs, NVCC_FLAGS),
                                                (OPS_LIB, _ops_sources, _ops_inputs, OPS_NVCC_FLAGS),
                                                (LAYER_LIB, _layer_sources, _layer_inputs,
                                                 OPS_NVCC_FLAGS))
            if force or _older(lib, inputs())]
    if not todo:
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(job):
        lib, src, flags = job
        obj = os.path.join(BUILD, {OPS_LIB: "ops_", LAYER_LIB: "layer_"}.get(lib, "") + os.path.basename(src) + ".o")
        cmd = [nvcc(), *flags, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return lib, obj, r.stderr

    objs = {}
    with concurrent.futures.ThreadPoolExecutor(max_workers=12) as ex:
        for lib, obj, log in ex.map(compile_one, [(lib, src, flags) for lib, srcs, flags in todo
                                                  for src in srcs]):
            objs.setdefault(lib, []).append(obj)
            if verbose and log:
                print(log)
    for lib, _, _ in todo:
        _link(objs[lib], lib)
    return LIB


def _link(objs, lib: str) -> None:
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=BUILD)
    os.close(fd)
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "lib64")
    r = subprocess.run([nvcc(), "-shared", "-cudart", "shared", *ARCH, *objs,
                        "-Xlinker", "-rpath", "-Xlinker", cuda_lib, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
