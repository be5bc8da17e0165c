"""Build the HIP library libdetgemm.so in-tree for gfx950 with hipcc, and the
torch extension module over it with the host compiler."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("detgemm.hip", "head.hip", "norm.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdetgemm.so")
# the benchmark's LDS-atomic peak probe: its own library, never loaded by the package
PROBE_SOURCES = [os.path.join(PKG, "csrc", "lds_probe.hip")]
PROBE_LIB = os.path.join(PKG, "liblds_probe.so")
# the torch side of the head operators (autograd, streams): host code only
OPS_SOURCE = os.path.join(PKG, "csrc", "head_ops.cpp")
OPS_LIB = os.path.join(PKG, "_ops.so")
ARCH = "gfx950"

# -packed-fp32-ops off: no v_pk_{add,mul,fma}_f32 in any generated code
HIPCC_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-shared", f"--offload-arch={ARCH}",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wall", "-Wno-unused-function", f"-I{INCLUDE}"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def _hipcc(sources, out: str, verbose: bool) -> str:
    cmd = [hipcc(), *HIPCC_FLAGS, f"-parallel-jobs={min(len(sources), 4)}", "-o", out + ".tmp", *sources]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in res.stderr.splitlines()
                    if "packed-fp32-ops" not in l and l.strip())
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err:
        print(err, file=sys.stderr)
    os.replace(out + ".tmp", out)
    return out


def _host_ops(verbose: bool) -> str:
    """Compile the torch extension module against libdetgemm.so (which must
    be built) and the installed torch."""
    from torch.utils.cpp_extension import include_paths, library_paths
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
           *[f"-I{p}" for p in (INCLUDE, *include_paths(), "/opt/rocm/include", sysconfig.get_paths()["include"])],
           "-o", OPS_LIB + ".tmp", OPS_SOURCE, f"-L{PKG}", "-l:libdetgemm.so",
           *[f"-L{p}" for p in library_paths()], "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed ({res.returncode}):\n{res.stderr}")
    os.replace(OPS_LIB + ".tmp", OPS_LIB)
    return OPS_LIB


def build(verbose: bool = False) -> str:
    """Build libdetgemm.so, the torch extension over it and the benchmark's
    probe library."""
    _hipcc(PROBE_SOURCES, PROBE_LIB, verbose)
    lib = _hipcc(SOURCES, LIB, verbose)
    _host_ops(verbose)
    return lib


def device_asm(out_path: str, source: str = SOURCES[0]) -> str:
    """Write the gfx950 assembly of one source's kernels (for inspection)."""
    cmd = [hipcc(), "-O3", "-std=c++17", f"--offload-arch={ARCH}", "--cuda-device-only", "-S",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", f"-I{INCLUDE}",
           "-o", out_path, source]
    subprocess.run(cmd, check=True, capture_output=True)
    return out_path


if __name__ == "__main__":
    print(build(verbose=True))
