"""Build libssm.so (the HIP kernels and the C ABI) in-tree for gfx950.

    python -m selective_state_space_fwd_amd.build

Every source is compiled with hipcc for gfx950 only.  Packed FP32 VALU
instructions are disabled with the target feature ``-packed-fp32-ops``; the
host pass prints a harmless warning that it does not know that feature.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = ROOT / "_build"
LIB = PKG / "libssm.so"
LAYER = PKG / "csrc_layer"
SOURCES = [CSRC / f for f in ("ssm_api.hip", "ssm_scan.hip", "ssm_tscan.hip", "ssm_update.hip",
                              "ssm_bwd.hip")]
SOURCES += [LAYER / f for f in ("layer_api.hip", "layer_heads.hip", "layer_heads_bf16.hip", "layer_heads_f32.hip",
                                "layer_heads_bwd.hip",
                                "layer_update.hip", "layer_conv.hip", "layer_norm.hip")]

ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}", f"-I{LAYER}",
]


def _compile(src: Path) -> Path:
    obj = BUILD / (src.stem + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", str(src), "-o", str(obj)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err:
        print(err, file=sys.stderr)
    return obj


def build() -> Path:
    """Compile every source and link libssm.so (always rebuilds)."""
    BUILD.mkdir(exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB.with_suffix(".so.tmp")
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *map(str, objs), "-o", str(tmp)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
