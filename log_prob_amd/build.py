"""Build libflce.so (HIP, gfx950 only) in-tree with hipcc, and its Python binding _binding.so.

    python -m log_prob_amd.build            # -> log_prob_amd/libflce.so, log_prob_amd/_binding.so
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["flce_kernels.hip", "norm_kernels.hip", "mx_quant_kernels.hip",
           "mx_stream_kernels.hip", "mx_tile_kernels.hip", "linear_kernels.hip",
           "logprob_kernels.hip", "dropout_kernels.hip", "flce_api.cpp", "ops_api.cpp",
           "block_api.cpp"]
LIB = os.path.join(HERE, "libflce.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed fp32 arithmetic is disabled for all device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def binding_needs() -> str:
    """What the Python binding's build lacks here; empty if it can be built."""
    torch = importlib.util.find_spec("torch")
    have = {"torch for ROCm": torch is not None and os.path.exists(os.path.join(
                torch.submodule_search_locations[0], "include", "c10", "hip", "HIPStream.h")),
            "g++": shutil.which("g++"),
            "Python.h": os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))}
    return " and ".join(name for name, there in have.items() if not there)


def compile_binding(obj: str, verbose: bool) -> str:
    """The binding's object file; returns torch's library folder."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    include = [os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           "-I", os.path.join(ROOT, "include"), *(f for d in include for f in ("-isystem", d)),
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return os.path.join(torch, "lib")


def link_binding(obj: str, torch_lib: str, lib_dir: str, out: str, verbose: bool) -> None:
    """Link against the libflce.so in lib_dir; at run time the one beside the binding is found."""
    cmd = ["g++", "-shared", obj, "-o", out, "-L", lib_dir, "-l:libflce.so", "-Wl,-rpath,$ORIGIN",
           "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10_hip", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def build(verbose: bool = False, extra_flags=(), out: str = LIB) -> str:
    """Build the library at `out`.  For the package's own one the compiled binding is built with
    it, or left out where torch or g++ is missing: its calls then go through ctypes.  Nothing is
    replaced before everything has been built."""
    cc = hipcc()
    bind = out == LIB
    if bind and binding_needs():
        print(f"without {binding_needs()} the Python binding is left out (calls go through ctypes)",
              flush=True)
    with_binding = bind and not binding_needs()
    with tempfile.TemporaryDirectory() as tmp:
        binding = os.path.join(tmp, "binding.o")
        def compile_one(src):
            obj = os.path.join(tmp, src + ".o")
            cmd = [cc, *HIPCC_FLAGS, *extra_flags, "-I", os.path.join(ROOT, "include"),
                   "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
            return obj

        # one compiler process a source, side by side
        with ThreadPoolExecutor(max_workers=min(len(SOURCES), 4)) as pool:
            torch_lib = pool.submit(compile_binding, binding, verbose) if with_binding else None
            objs = list(pool.map(compile_one, SOURCES))
        lib = os.path.join(tmp, "libflce.so")
        cmd = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", lib]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        if with_binding:
            link_binding(binding, torch_lib.result(), tmp, BINDING + ".tmp", verbose)
        shutil.copy(lib, out + ".tmp")
    os.replace(out + ".tmp", out)
    if with_binding:
        os.replace(BINDING + ".tmp", BINDING)
    elif bind and os.path.exists(BINDING):
        os.remove(BINDING)   # it was built with another library
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
