"""Build libfp8bs.so (HIP, gfx950 only) in-tree with hipcc.

    python -m fp8_block_scaled_x128_amd.build [--resource-usage]

Every source is compiled for gfx950 with -ffp-contract=off (the kernels place
their FMAs explicitly) and with packed-FP32 code generation disabled.
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfp8bs.so")
SOURCES = ["quant.hip", "gemm.hip", "moe.hip", "norm.hip", "norm_bwd.hip", "route.hip", "route_grouped.hip", "int8_quant.hip", "int8_gemm.hip", "capi.hip"]
# The GEMM promotes MFMA results with VALU FMAs, so the results must land in
# VGPRs (not AGPRs, which would need a v_accvgpr_read per value).
EXTRA = {"gemm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}
# Kernels whose inline assembly names accumulation registers of its own choice: the
# compiler must keep its values and spills out of them (check_accumulators).
OWN_ACCUMULATORS = {"int8_gemm.hip": r"k_i8_tile(_pair)?ILi4ELi4E"}
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"), "-Wall", "-Wno-unused-function"]


def check_accumulators(listing: str, kernels: str) -> None:
    """Raise where a kernel of an assembly listing whose name matches `kernels` uses an
    accumulation register outside of inline assembly, or where there is no such kernel."""
    name, own, found = None, False, 0
    for line in listing.splitlines():
        label = re.match(r"(\w+):", line)
        if label:
            name = label.group(1) if re.search(kernels, label.group(1)) else None
            own = False
            found += name is not None
        elif line.startswith(".Lfunc_end"):
            name = None
        elif "#ASMSTART" in line or "#ASMEND" in line:
            own = "#ASMSTART" in line
        elif name and not own and re.search(r"\ba(\d+\b|\[\d+(:\d+)?\])", line.split(";")[0]):
            raise RuntimeError("%s: the compiler uses an accumulation register of the kernel's own: %s" % (name, line.strip()))
    if not found:
        raise RuntimeError("no kernel matches %s" % kernels)


def _check_listing(src: str) -> str:
    """check_accumulators of the code compiled from one source."""
    out = os.path.join(ROOT, "_build", os.path.basename(src).replace(".hip", ".s"))
    log = _compile(src, out, ["--cuda-device-only", "-S"] + EXTRA.get(os.path.basename(src), []))
    with open(out) as f:
        check_accumulators(f.read(), OWN_ACCUMULATORS[os.path.basename(src)])
    return log


def _compile(src: str, obj: str, extra):
    cmd = [HIPCC, *FLAGS, *(["-c"] if "-S" not in extra else []), *extra, src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                    if "packed-fp32-ops" not in l and "not a recognized feature" not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, out))
    return out


def build(resource_usage: bool = False, verbose: bool = False) -> str:
    """Compile every HIP source and link libfp8bs.so; returns its path."""
    bdir = os.path.join(ROOT, "_build")
    os.makedirs(bdir, exist_ok=True)
    extra = ["-Rpass-analysis=kernel-resource-usage"] if resource_usage else []
    objs = [os.path.join(bdir, s.replace(".hip", ".o")) for s in SOURCES]
    with ThreadPoolExecutor(len(SOURCES) + len(OWN_ACCUMULATORS)) as ex:
        checks = [ex.submit(_check_listing, os.path.join(CSRC, s)) for s in OWN_ACCUMULATORS]
        outs = list(ex.map(lambda so: _compile(os.path.join(CSRC, so[0]), so[1], extra + EXTRA.get(so[0], [])),
                           zip(SOURCES, objs)))
        for c in checks:
            c.result()
    if verbose or resource_usage:
        for o in outs:
            if o.strip():
                print(o)
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.check_call([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(resource_usage="--resource-usage" in sys.argv, verbose="-v" in sys.argv))
