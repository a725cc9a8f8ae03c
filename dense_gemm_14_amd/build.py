"""Build libgemm355.so in-tree with hipcc for gfx950 (no GPU needed to compile),
and the binding's _marshal module with gcc."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libgemm355.so")
SOURCES = [os.path.join(CSRC, f) for f in ("gemm355.hip", "dense_ops.hip", "loss_ops.hip", "model_ops.hip")]
HEADERS = [os.path.join(CSRC, f) for f in ("common.hpp", "gemm_bf16.hpp", "gemm_bf16_small.hpp", "gemm_bf16_small_long.hpp", "gemm_bf16_splitk.hpp",
                                           "gemm_fp4.hpp", "fp4_decode.hpp", "gemm_mxfp4.hpp", "schedule.hpp", "host.hpp",
                                           "dense_common.hpp", "dense_large.hpp", "dense_small.hpp", "dense_tile.hpp", "dense_grad.hpp", "newton_schulz.hpp",
                                           "checks.hpp", "dense_plan.hpp", "dense_loss.hpp", "cross_entropy.hpp", "vector8.hpp", "embedding.hpp", "layer_norm.hpp")] + \
    [os.path.join(INCLUDE, "gemm355.h")]

MARSHAL_SOURCE = os.path.join(CSRC, "marshal.c")
# (the tag keeps another interpreter from loading it)
MARSHAL_PATH = os.path.join(HERE, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # the LDS copies clobber m0 on purpose (the compiler uses m0 nowhere else)
    "-Wno-inline-asm",
    # packed FP32 instructions stay off: the compiler must not form them
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _hipcc(args, verbose):
    cmd = [HIPCC, *args]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = ("packed-fp32-ops", "unknown target feature")
    msgs = [l for l in (res.stdout + res.stderr).splitlines() if l and not any(n in l for n in noise)]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed (%d):\n%s" % (res.returncode, "\n".join(msgs)))
    if msgs and verbose:
        print("\n".join(msgs), file=sys.stderr)


def build_marshal() -> str:
    out = MARSHAL_PATH + ".tmp%d" % os.getpid()
    res = subprocess.run(["gcc", "-O2", "-Wall", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-o", out,
                          MARSHAL_SOURCE], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("gcc failed (%d):\n%s" % (res.returncode, res.stdout + res.stderr))
    os.replace(out, MARSHAL_PATH)
    return MARSHAL_PATH


def build(verbose: bool = False) -> str:
    """Compile every HIP source of the library into LIB_PATH, and the binding's
    marshalling. Always recompiles."""
    build_marshal()
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:   # one compiler process per source
            list(pool.map(lambda so: _hipcc([*FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", so[1], so[0]], verbose),
                          zip(SOURCES, objs)))
        out = LIB_PATH + ".tmp%d" % os.getpid()
        _hipcc(["--offload-arch=gfx950", "-shared", "-fPIC", "-o", out, *objs], verbose)
    os.replace(out, LIB_PATH)
    return LIB_PATH


def stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(MARSHAL_PATH):
        return True
    if os.path.getmtime(MARSHAL_SOURCE) > os.path.getmtime(MARSHAL_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(s) > t for s in SOURCES + HEADERS)


if __name__ == "__main__":
    print(build(verbose=True))
