"""Build libhgemm.so (the C-ABI library with its gfx950 kernels) in-tree.

    python half_precision_gemm_amd/build.py          # or __graft_entry__.build()

hipcc cross-compiles for gfx950 without a GPU.  Packed-fp32 VALU ops are
disabled for all device code (-packed-fp32-ops feature off).
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libhgemm.so")
SOURCES = [os.path.join(CSRC, "hg_api.cpp"), os.path.join(CSRC, "hg_kernels.hip"),
           os.path.join(CSRC, "hg_fast.hip"), os.path.join(CSRC, "hg_ring.hip"),
           os.path.join(CSRC, "hg_trsm.hip"), os.path.join(CSRC, "hg_xform.hip"),
           os.path.join(CSRC, "hg_noalloc.hip"), os.path.join(CSRC, "hg_linear_api.cpp"),
           os.path.join(CSRC, "hg_linear_ring.hip"), os.path.join(CSRC, "hg_linear_rows.hip"),
           os.path.join(CSRC, "hg_linear_tile.hip"), os.path.join(CSRC, "hg_linear_rowwise.hip"),
           os.path.join(CSRC, "hg_linear_loose.hip"), os.path.join(CSRC, "hg_linear_outer.hip")]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc failed building libhgemm.so")


def build(extra=(), out=LIB, verbose=False):
    """Compiles every source (several at a time) and links them into `out`."""
    tmp = out + ".tmp%d" % os.getpid()
    jobs = min(8, int(os.environ.get("MAX_JOBS", 0)) or os.cpu_count() or 1)
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(jobs) as pool:
            list(pool.map(lambda so: _run([HIPCC] + FLAGS + list(extra) + ["-c", so[0], "-o", so[1]], verbose),
                          zip(SOURCES, objs)))
        _run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared"] + list(extra) + ["-o", tmp] + objs, verbose)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
