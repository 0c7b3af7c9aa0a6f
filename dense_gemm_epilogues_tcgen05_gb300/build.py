"""Build the CUDA library in-tree: csrc/*.cu -> libgemm_gb300.so (sm_103a only).

Each translation unit is compiled by its own nvcc process (in parallel), then
linked into one shared library next to this file, against the shared CUDA
runtime (so a process that already loaded PyTorch's runtime reuses it).
Object files and ptxas reports go to ``_build/`` at the repository root.

Usage:  python dense_gemm_epilogues_tcgen05_gb300/build.py [--force] [-v]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import hashlib
import os
import re
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO, "include")
BUILD_DIR = os.path.join(REPO, "_build")
LIB_NAME = "libgemm_gb300.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH_FLAGS + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xptxas", "-v", "-DNDEBUG",
]


# Kernels whose warpgroups trade registers (setmaxnreg): the trade adds up for this count at launch and no other,
# and a sum above what the block was launched with would wait for ever.
LAUNCH_REGISTERS = {"i8_tc_kernel": 72}


def check_registers(report: str) -> None:
    """Raise unless the compiler gave every kernel of LAUNCH_REGISTERS the count that its source is written for."""
    for name, want in LAUNCH_REGISTERS.items():
        got = [int(m.group(1)) for part in report.split("Compiling entry function")[1:]
               if name in part.split("'")[1] for m in [re.search(r"Used (\d+) registers", part)] if m]
        if not got or any(r != want for r in got):
            raise RuntimeError(f"{name}: compiled to {sorted(set(got)) or 'no'} registers, written for {want}; its "
                               f"source's LAUNCH_REGS and register trade need to follow this compiler")


def _nvcc() -> str:
    cand = [os.environ.get("NVCC", ""), shutil.which("nvcc") or "", "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found (CUDA toolkit required to build the library)")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def source_fingerprint() -> str:
    """Hash of every kernel / header source and the nvcc flags (machine-independent:
    profile records taken on the GPU host are matched against it)."""
    h = hashlib.sha256()
    for d in (CSRC, INCLUDE):
        for f in sorted(os.listdir(d)):
            p = os.path.join(d, f)
            if os.path.isfile(p):
                h.update(f.encode())
                with open(p, "rb") as fh:
                    h.update(fh.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()


def _fingerprint() -> str:
    return source_fingerprint() + "-" + os.uname().machine


def _compile(nvcc: str, src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc] + NVCC_FLAGS + ["-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    log = r.stdout + r.stderr
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{log}")
    return obj, log


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if any source changed; returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp = os.path.join(BUILD_DIR, "stamp.txt")
    fp = _fingerprint()
    if not force and os.path.exists(LIB_PATH) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == fp:
                return LIB_PATH
    nvcc = _nvcc()
    srcs = _sources()
    logs = []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        futs = {ex.submit(_compile, nvcc, s): s for s in srcs}
        objs = []
        for fut in cf.as_completed(futs):
            obj, log = fut.result()
            objs.append(obj)
            logs.append(log)
    with open(os.path.join(BUILD_DIR, "ptxas_report.txt"), "w") as f:
        f.write("\n".join(logs))
    check_registers("\n".join(logs))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc] + ARCH_FLAGS + ["-shared", "-o", tmp] + sorted(objs) + [
        "-cudart", "shared", "-Xlinker", "-rpath,$ORIGIN:/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB_PATH)
    with open(stamp, "w") as f:
        f.write(fp)
    if verbose:
        print("\n".join(logs))
    return LIB_PATH


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
