"""Build libselscan.so in-tree for gfx950 with hipcc (cross-compiles without a GPU).

    python -m selective_state_space_43_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SRCS = [os.path.join(CSRC, n) for n in ("selscan.hip", "mixer.hip")]
OUT = os.path.join(HERE, "libselscan.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed-FP32 VALU forms are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA accumulators in ordinary VGPRs: the Mamba-2 scan scales and splits
    # its state between products, which AGPRs would turn into copies
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmds, verbose):
    """Runs the commands side by side; raises with what a failing one printed."""
    # hipcc's host pass does not know the device-only feature name; that note is harmless
    noise = "'-packed-fp32-ops' is not a recognized feature"
    if verbose:
        for cmd in cmds:
            print(" ".join(cmd), flush=True)
    procs = [subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for cmd in cmds]
    said = [p.communicate()[0] for p in procs]
    for p, text in zip(procs, said):
        msgs = [ln for ln in text.splitlines() if noise not in ln and ln.strip()]
        if p.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
        if verbose and msgs:
            print("\n".join(msgs))


def build(verbose: bool = False) -> str:
    tmp = OUT + ".tmp%d" % os.getpid()
    objs = [tmp + "." + os.path.basename(src)[:-4] + ".o" for src in SRCS]
    try:
        _run([[HIPCC, *FLAGS, "-c", "-o", obj, src] for obj, src in zip(objs, SRCS)], verbose)
        _run([[HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]], verbose)
        os.replace(tmp, OUT)
    finally:
        for path in (tmp, *objs):
            if os.path.exists(path):
                os.remove(path)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
