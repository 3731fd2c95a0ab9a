"""Build libfno.so (the HIP kernels and the C ABI) for gfx950 with hipcc.

    python -m spectral_convolution_amd.build        # or build() from Python

Objects go to spectral_convolution_amd/_build/, the library next to this file.
Every HIP translation unit is compiled with packed-fp32 instructions disabled.
"""

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfno.so")
NATIVE = os.path.join(HERE, "_native.so")

SOURCES = ["plane_kernels.hip", "plane_mfma.hip", "axis_kernels.hip", "contract.hip", "contract_mx.hip", "backward.hip", "weights.hip", "pointwise.hip", "fused.hip", "fno_api.cpp",
           "fno_model.cpp", "checkpoint.hip", "norm.hip", "norm_f32.hip", "norm_f16.hip", "norm_bf16.hip", "mix_train.hip", "mix_train_f16.hip", "mix_train_bf16.hip",
           "fno_train.cpp"]
HEADERS = ["common.hpp", "fft_reg.hpp", "plane_common.hpp", "plane_valu.hpp", "plane_mfma.hpp", "contract.hpp", "train.hpp", "checkpoint.hpp", "gelu.hpp", "mix_train.hpp", "mix_train_half.hpp", "norm_common.hpp", "norm_field.hpp", "norm_token.hpp"]

ARCH = "gfx950"
CFLAGS = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unknown-pragmas",
    "-I", os.path.join(ROOT, "include"),
]


def _hipcc():
    h = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(h):
        raise RuntimeError("hipcc not found; the HIP library cannot be built")
    return h


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc(), "-x", "hip", *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _native(verbose):
    """Compile the binding's own extension (host code against torch's headers).
    Where torch is not installed the binding has no use either, and libfno.so needs neither."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        print("torch is not installed: _native.so, the extension of the Python binding, is not built", file=sys.stderr)
        return
    torch = os.path.dirname(spec.origin)
    tmp = NATIVE + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-I", os.path.join(torch, "include"), "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(torch, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)


def build(verbose: bool = False, jobs: int = 8) -> str:
    """Compile every source, link libfno.so and build the binding's extension;
    returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        native = ex.submit(_native, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    native.result()  # its failure is reported once the library is there
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
