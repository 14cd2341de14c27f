"""Build libzero_mi355x.so (the C-ABI HIP library) in-tree for gfx950.

Flags that matter for the numerics:
  -ffp-contract=off                         no a*b+c -> fma contraction, so every
                                            operation rounds once, as specified;
  -fhip-fp32-correctly-rounded-divide-sqrt  IEEE division and square root;
  (default)                                 fp32/fp16 denormals are kept.
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                            keep the compiler from forming packed
                                            fp32 arithmetic.
The host-only C++ sources are compiled by ROCm's clang++ as plain C++ (no
device pass), with the same no-contraction rule, and linked into the same
library.
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libzero_mi355x.so")
SOURCES = ["host.hip", "flatten.hip", "norm.hip", "adam.hip", "onebit.hip", "dropout.hip", "layernorm.hip",
           "layernorm_bwd.hip"]
HOST_SOURCES = ["host_step.cpp"]          # plain C++ (the CPU side of the offloaded step)
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if c and os.path.exists(c):
            return c
    return "hipcc"


HOST_FLAGS = ["-x", "c++", "-std=c++17", "-O3", "-fPIC", "-ffp-contract=off", "-Wall",
              "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"]


def host_cxx() -> str:
    for c in (os.environ.get("ZERO_HOST_CXX"), "/opt/rocm/llvm/bin/clang++"):
        if c and os.path.exists(c):
            return c
    return "clang++"


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile every source into the in-tree shared library (always rebuilds),
    the sources side by side."""
    tmp = LIB + ".tmp"
    common = [f"-I{INCLUDE}", f"-I{CSRC}"]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    with tempfile.TemporaryDirectory() as objdir:
        obj = lambda src: os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
        cmds = [[hipcc(), *compile_flags, *extra_flags, *common, "-c", os.path.join(CSRC, src), "-o", obj(src)]
                for src in SOURCES]
        cmds += [[host_cxx(), *HOST_FLAGS, *common, "-c", os.path.join(CSRC, src), "-o", obj(src)]
                 for src in HOST_SOURCES]
        with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as pool:
            list(pool.map(run, cmds))
        run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp,
             *[obj(src) for src in SOURCES + HOST_SOURCES], "-lpthread"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
