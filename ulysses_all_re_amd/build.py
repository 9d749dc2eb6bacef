"""Build the in-tree HIP library ulysses_all_re_amd/libua2a.so for gfx950.

    python -m ulysses_all_re_amd.build

The library is compiled with hipcc for MI355X (gfx950) only, from the
sources under csrc/ and the public header include/ua2a.h.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libua2a.so")
SOURCES = [os.path.join(CSRC, "ua2a_kernels.hip"), os.path.join(CSRC, "ua2a_host.cpp"),
           os.path.join(CSRC, "ua2a_act_norm.hip"), os.path.join(CSRC, "ua2a_act_norm_grad.hip"),
           os.path.join(CSRC, "ua2a_act_cache.hip"), os.path.join(CSRC, "ua2a_act_launch.hip"),
           os.path.join(CSRC, "ua2a_act_host.cpp")]
HEADERS = [os.path.join(INCLUDE, "ua2a.h"), os.path.join(INCLUDE, "ua2a_act.h"),
           os.path.join(CSRC, "ua2a_geometry.h"), os.path.join(CSRC, "ua2a_bodies.h"),
           os.path.join(CSRC, "ua2a_internal.h"), os.path.join(CSRC, "ua2a_act_geometry.h"),
           os.path.join(CSRC, "ua2a_act_internal.h"), os.path.join(CSRC, "ua2a_act_device.h"),
           os.path.join(CSRC, "ua2a_act_norm.h")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Werror",
    "-Wno-unused-command-line-argument",
    # keep the compiler from forming packed-fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]


def build(verbose: bool = False) -> str:
    """Compile libua2a.so (always recompiles) and return its path.  The
    sources are compiled side by side, then linked."""
    tmp = f"{LIBRARY}.tmp{os.getpid():x}"
    with tempfile.TemporaryDirectory() as work:
        jobs, objects = [], []
        for src in SOURCES:
            obj = os.path.join(work, os.path.basename(src) + ".o")
            objects.append(obj)
            cmd = [HIPCC, *FLAGS, "-c", "-x", "hip", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append((cmd, subprocess.Popen(cmd)))
        failed = [cmd for cmd, job in jobs if job.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        cmd = [HIPCC, *FLAGS, "-shared", *objects, "-o", tmp]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
