"""Builds libdwpt_scan.so (the HIP kernels and the C ABI) for gfx950 with hipcc."""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")          # the scans
CSRC_SEQ = os.path.join(PKG_DIR, "csrc_seq")  # the sequence-model operators
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libdwpt_scan.so")
ARCH = "gfx950"

HIPCC_FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-shared",
    # no packed-FP32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC_SEQ, "*.hip")))


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msg = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed (%d):\n%s\ncommand: %s" % (res.returncode, msg, " ".join(cmd)))
    return msg


def _compile(flags, srcs, out):
    """Compiles every source into an object of its own, side by side, and links them into `out`."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    compile_flags = [f for f in flags if f != "-shared"] + ["-I" + INCLUDE, "-I" + CSRC, "-I" + CSRC_SEQ, "-c"]
    tmp = out + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, "%d.o" % i) for i in range(len(srcs))]
        with ThreadPoolExecutor(max(1, min(len(srcs), (os.cpu_count() or 2) // 2))) as pool:
            msgs = list(pool.map(lambda so: _run([hipcc] + compile_flags + [so[0], "-o", so[1]]), zip(srcs, objs)))
        try:
            # device code is complete in every object: the link is the host's
            msgs.append(_run([hipcc] + flags + objs + ["-o", tmp]))
            os.replace(tmp, out)
        finally:
            if os.path.exists(tmp):
                os.remove(tmp)
    return "\n".join(m for m in msgs if m.strip())


def build(verbose: bool = False) -> str:
    """Compile every source into one shared library; always recompiles."""
    msg = _compile(HIPCC_FLAGS, sources(), LIB_PATH)
    if verbose and msg:
        print(msg)
    return LIB_PATH


def build_asan(driver: str, out: str, verbose: bool = False) -> str:
    """The library's sources and a test driver (C++ calling the C ABI) as one executable
    whose host code is built with AddressSanitizer (device code as in the library)."""
    flags = [f for f in HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-g"]
    msg = _compile(flags + san, sources() + [driver], out)
    if verbose and msg:
        print(msg)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
