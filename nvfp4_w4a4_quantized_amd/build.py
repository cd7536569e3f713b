"""Build libnvfp4.so (the C ABI + HIP kernels) for gfx950 with hipcc, in-tree, and
_torch_binding.so (host code: torch tensors to the C ABI) against it.

Each source is compiled to an object in its own process (in parallel), then the
objects are linked into the shared libraries.  Every call rebuilds everything.  The
library needs hipcc alone; the binding needs g++, Python's headers and torch, and without
torch it is left out.

    python nvfp4_w4a4_quantized_amd/build.py

It imports nothing from the package, whose import needs the built library.
"""

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnvfp4.so")
BINDING = os.path.join(HERE, "_torch_binding.so")
OBJDIR = os.path.join(ROOT, "_build")

SOURCES = ["abi.cpp", "quant.hip", "gemm.hip", "gemv.hip", "skinny.hip", "requant.hip", "mx.hip", "noalloc.hip", "gdn.hip", "probe.hip", "soloq.hip", "kvcache.hip",
           "kvattn.hip", "kvprefill.hip"]

COMPILE_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++20",
    "-fPIC",
    "-fvisibility=hidden",
    # the quantizer relies on exactly rounded float64/fp32 operations: no contraction
    "-ffp-contract=off",
    # keep the compiler from forming packed-fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]
LINK_FLAGS = ["--offload-arch=gfx950", "-shared", "-fPIC"]
BINDING_SOURCE = "torch_binding.cpp"


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(os.path.basename(cmd[0]) + " failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)


def _binding_commands():
    """Compile and link of the host-only binding (None without torch).  torch is found, not
    imported; its libraries are loaded by the time the binding is."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    torch = os.path.dirname(spec.origin)
    obj = os.path.join(OBJDIR, "torch_binding.o")
    compile_ = ["g++", "-O2", "-std=c++20", "-fPIC", "-fvisibility=hidden", "-w", "-isystem",
                os.path.join(torch, "include"), "-I", sysconfig.get_paths()["include"], "-c", "-o", obj,
                os.path.join(CSRC, BINDING_SOURCE)]
    link = ["g++", "-shared", "-o", BINDING + ".tmp", obj, "-L" + HERE, "-lnvfp4", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    return compile_, link


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    os.makedirs(OBJDIR, exist_ok=True)
    objs = [os.path.join(OBJDIR, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    cmds = [[hipcc] + COMPILE_FLAGS + ["-c", "-o", o, os.path.join(CSRC, s)] for s, o in zip(SOURCES, objs)]
    binding = _binding_commands()
    with ThreadPoolExecutor(max_workers=len(cmds) + 1) as ex:
        compiled = ex.submit(_run, binding[0], verbose) if binding else None
        for f in [ex.submit(_run, c, verbose) for c in cmds]:
            f.result()
    tmp = LIB + ".tmp"
    _run([hipcc] + LINK_FLAGS + ["-o", tmp] + objs, verbose)
    os.replace(tmp, LIB)
    # the library stands by itself: it is there whatever becomes of the binding
    if binding is None:
        print("torch is not installed: _torch_binding.so is not built", file=sys.stderr)
        return LIB
    compiled.result()
    _run(binding[1], verbose)
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
