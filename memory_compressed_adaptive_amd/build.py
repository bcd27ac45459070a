"""Builds the package's native libraries in-tree with hipcc for gfx950.

    python -m memory_compressed_adaptive_amd.build

libmicroadam.so  -- the MicroAdam step, the Muon operators and AdamW over
                    many tensors (C ABI in include/microadam.h)
_tensors.so      -- reads lists of torch tensors into the arrays of the calls that
                    take many (host code, built against torch's headers)
libmasynth.so    -- the seeded synthetic-input generator used by the benchmark
                    and the tests (no optimizer arithmetic in it)

Floating point: no contraction (fp32 results must equal the CPU oracle's one
rounding per operation), correctly rounded fp32 division and square root,
denormals kept, and no packed-fp32 instructions.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result", "-Wno-unused-function", "-Wno-unused-value",
    f"-I{INCLUDE}", f"-I{CSRC}",
]

TARGETS = {
    "libmicroadam.so": [os.path.join(CSRC, "microadam.hip"), os.path.join(CSRC, "muon.hip"),
                        os.path.join(CSRC, "adamw_many.hip")],
    "libmasynth.so": [os.path.join(CSRC, "synth.hip")],
}


EXTENSION = "_tensors.so"


def _extension_command(dst: str) -> list[str]:
    """Host code only."""
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    include = [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"),
               *cpp_extension.include_paths()]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            "-D__HIP_PLATFORM_AMD__=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
            *(x for d in include for x in ("-isystem", d)), os.path.join(CSRC, "tensors.cpp"), "-o", dst,
            f"-L{lib}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {what}")
    if verbose and r.stderr.strip():
        # hipcc's host pass does not know the packed-fp32 feature; harmless
        lines = [ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln]
        if any(ln.strip() for ln in lines):
            sys.stderr.write("\n".join(lines) + "\n")


def build(verbose: bool = False, only: str | None = None) -> list[str]:
    """Compiles every source to an object (all at once), then links each library."""
    out = []
    targets = {name: srcs for name, srcs in TARGETS.items() if not only or name == only}
    with tempfile.TemporaryDirectory() as tmpdir, ThreadPoolExecutor() as pool:
        obj = {src: os.path.join(tmpdir, os.path.basename(src) + ".o") for srcs in targets.values() for src in srcs}
        jobs = [pool.submit(_run, [HIPCC, *COMMON, "-c", src, "-o", o], src, verbose) for src, o in obj.items()]
        if not only or only == EXTENSION:
            dst = os.path.join(PKG, EXTENSION)
            _run(_extension_command(dst + ".tmp"), EXTENSION, verbose)
            os.replace(dst + ".tmp", dst)
            out.append(dst)
        for job in jobs:
            job.result()
        for name, srcs in targets.items():
            dst = os.path.join(PKG, name)
            tmp = dst + ".tmp"
            _run([HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", *(obj[src] for src in srcs), "-o", tmp], name, verbose)
            os.replace(tmp, dst)
            out.append(dst)
    return out


if __name__ == "__main__":
    for p in build(verbose="-v" in sys.argv):
        print(p)
