"""Build libtara_attn.so in-tree with nvcc for sm_100a.

    python -m video_diffusion_attention_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libtara_attn.so")
# the same sources with the kernels' device-side checks compiled in (-DTARA_DEBUG=1)
LIB_DEBUG = os.path.join(LIB_DIR, "libtara_attn_debug.so")
SOURCES = [os.path.join(CSRC, f) for f in
           ("tara_abi.cu", "tara_layer.cu", "tara_pack.cpp", "tara_host.cpp")]
HEADERS = [os.path.join(ROOT, "include", "tara_attn.h")] + [
    os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cuh", ".h"))]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "-cudart", "static",
    "--expt-relaxed-constexpr",
]

# Kernels that redistribute registers among their warps draw on exactly the number per thread
# that their source states: the library refuses to launch them with any other.
SPLIT_KERNELS = {"attn_tc_kernel": ("attn_tc.cuh", "kTcLaunchRegs"),
                 "attn_pair_kernel": ("attn_tc.cuh", "kTcLaunchRegs"),
                 "linear_pair_kernel": ("linear_pair.cuh", "kPairLinRegs")}


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in SOURCES + HEADERS)


def split_registers() -> dict:
    """{kernel: registers per thread its source counts on}."""
    want = {}
    for kernel, (header, name) in SPLIT_KERNELS.items():
        with open(os.path.join(CSRC, header)) as f:
            want[kernel] = int(re.search(r"constexpr int %s = (\d+);" % name, f.read()).group(1))
    return want


def check_registers(ptxas_log: str, want: dict) -> int:
    """Raises when ptxas gave an instantiation of one of the kernels another number of registers;
    returns how many instantiations there are."""
    seen, entry = 0, ""
    for line in ptxas_log.splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            entry = m.group(1)
        m = re.search(r"Used (\d+) registers", line)
        if not m or not entry:
            continue
        for kernel, regs in want.items():
            # the name as a whole, in its mangled form
            if "%d%s" % (len(kernel), kernel) in entry:
                seen += 1
                if int(m.group(1)) != regs:
                    raise RuntimeError(
                        "ptxas gave %s %s registers a thread where its register split counts on "
                        "%d: another compiler needs another split (%s in csrc/%s)" %
                        ((entry, m.group(1), regs) + SPLIT_KERNELS[kernel][::-1]))
        entry = ""
    return seen


def build(force: bool = False, verbose_ptxas: bool = False, debug: bool = False) -> str:
    """Compile the release library (or, with debug=True, libtara_attn_debug.so with the
    kernels' device-side checks) if a source is newer than it or force is set.  The translation
    units are compiled side by side."""
    lib = LIB_DEBUG if debug else LIB
    if not force and not stale(lib):
        return lib
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = lib + ".tmp%d" % os.getpid()
    base = [nvcc()] + NVCC_FLAGS + ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if debug:
        base += ["-DTARA_DEBUG=1"]
    want = split_registers()

    def compile_unit(src: str, obj: str) -> int:
        p = subprocess.run(base + ["-Xptxas", "-v", "-c", "-o", obj, src],
                           stderr=subprocess.PIPE, text=True)
        if verbose_ptxas or p.returncode != 0:
            sys.stderr.write(p.stderr)
        else:   # warnings, without what -v adds
            sys.stderr.write("".join(
                line for line in p.stderr.splitlines(True)
                if not re.match(r"ptxas info|\s+\d+ bytes stack frame", line)))
        if p.returncode != 0:
            raise subprocess.CalledProcessError(p.returncode, p.args)
        return check_registers(p.stderr, want)

    with tempfile.TemporaryDirectory(dir=LIB_DIR) as work:
        objs = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
            if sum(pool.map(compile_unit, SOURCES, objs)) == 0:
                raise RuntimeError("ptxas reported no register counts")
        subprocess.check_call([nvcc()] + NVCC_FLAGS + ["-shared", "-o", tmp] + objs)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv,
                debug="--debug" in sys.argv))
