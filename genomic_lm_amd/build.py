"""Build libhyena.so for gfx950 in-tree (genomic_lm_amd/libhyena.so).

Every .hip / .cpp file under csrc/ is compiled with hipcc to an object, in
parallel, then linked into one shared library.  Run as
``python -m genomic_lm_amd.build`` or through ``__graft_entry__.build()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhyena.so")
ARCH = os.environ.get("HYENA_ARCH", "gfx950")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC)")


def flags() -> list[str]:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        "-I", INCLUDE, "-I", CSRC,
        # packed fp32 instructions off for all device code
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wno-unused-command-line-argument",
    ]


# Extra flags per source file.  The MFMA kernels keep their accumulators in
# ordinary VGPRs: the AGPR form costs a v_accvgpr_read for every result
# element used by the vector ALUs, and in the FFT kernels, which generate h
# on the matrix cores, its 32 AGPRs would come on top of the 128 registers
# that four waves per SIMD leave each wave.
EXTRA_FLAGS = {
    "attn_narrow.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "attn_wide.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "chunk_mfma.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "fftconv.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "linear_dma.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "linear_few.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "linear_tile.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "fir_mfma.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
}


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".hip", ".cpp")))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc(), *flags(), *EXTRA_FLAGS.get(os.path.basename(src), []), "-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB} from {len(srcs)} sources")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
