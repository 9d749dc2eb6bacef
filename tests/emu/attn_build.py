"""Build the host emulation of the attention operators (tests only):
libua2a_attn_emu.so = the library's own host code of ua2a_attn.h and ua2a.h with
a backend that carries out the launches on host memory (attn_backend.cpp)."""
from __future__ import annotations

import os
import subprocess

from tests.emu.build import CSRC, HERE, ROOT

SOURCES = [os.path.join(HERE, "attn_backend.cpp"), os.path.join(CSRC, "ua2a_attn_host.cpp"),
           os.path.join(CSRC, "ua2a_host.cpp")]
HEADERS = [os.path.join(CSRC, h) for h in ("ua2a_attn_geometry.h", "ua2a_attn_internal.h", "ua2a_act_geometry.h",
                                           "ua2a_act_internal.h", "ua2a_act_checks.h", "ua2a_geometry.h",
                                           "ua2a_internal.h")]
HEADERS += [os.path.join(ROOT, "include", h) for h in ("ua2a.h", "ua2a_act.h", "ua2a_attn.h")]
LIBRARY = os.path.join(HERE, "libua2a_attn_emu.so")


def build() -> str:
    """The library's path, compiled again if a source is newer."""
    if os.path.exists(LIBRARY) and all(os.path.getmtime(s) <= os.path.getmtime(LIBRARY) for s in SOURCES + HEADERS):
        return LIBRARY
    tmp = f"{LIBRARY}.tmp{os.getpid():x}"
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-g", "-fPIC", "-shared", "-Wall", "-Wextra", "-Werror",
                           "-Wno-unused-parameter", "-Wno-unknown-pragmas", "-D__HIP_PLATFORM_AMD__",
                           "-I/opt/rocm/include", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *SOURCES,
                           "-o", tmp])
    os.replace(tmp, LIBRARY)
    return LIBRARY
