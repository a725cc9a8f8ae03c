"""The host half of the library compiled without optimisation and with a trap at
whatever C++ leaves undefined (a division by zero, a sum beyond its type, arithmetic on
no pointer, a shift too far), in a process of its own against the stand-in for the HIP
runtime: the size queries of the embedding, layer norm and cross entropy calls over
their whole range, and every launch of those and of the layer calls."""
import ctypes
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from dense_gemm_14_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
TOP = (1 << 31) - 1


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    """(the stand-in, the library's host half)."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("needs hipcc")
    d = str(tmp_path_factory.mktemp("host"))
    run = lambda *a: subprocess.run(a, check=True, capture_output=True, text=True)
    shim, lib = os.path.join(d, "recorder.so"), os.path.join(d, "host.so")
    run("gcc", "-O1", "-Wall", "-shared", "-fPIC", "-o", shim, os.path.join(HERE, "launch_recorder.c"))
    objs = [os.path.join(d, os.path.basename(s) + ".o") for s in build.SOURCES]

    def compile_one(source, obj):
        run(build.HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O0", "-std=c++17", "-fPIC", "-w", "-Xarch_host",
            "-fsanitize=undefined", "-Xarch_host", "-fsanitize-trap=undefined", "-I", build.INCLUDE, "-I", build.CSRC, "-c",
            "-o", obj, source)
    with ThreadPoolExecutor(len(objs)) as pool:
        list(pool.map(compile_one, build.SOURCES, objs))
    # (what the device's code would be linked in by)
    code = sorted(set(re.findall(r"__hip_fatbin_[0-9a-f]+", run("nm", "-u", *objs).stdout)))
    run(build.HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib, *objs, *["-Wl,--defsym=%s=0" % c for c in code])
    return shim, lib


def child(what, shim, lib, *args):
    p = subprocess.run([sys.executable, "-X", "faulthandler", "-m", "tests.test_host_undefined", what, shim, lib, *args],
                       cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, "%d: %s %s" % (p.returncode, p.stdout[-2000:], p.stderr[-3000:])
    return p.stdout.split()


def near(*limits):
    """Sizes around these, and over the whole range."""
    s = {v + d for v in (*limits, *(1 << i for i in range(31)), TOP) for d in (-8, -1, 0, 1, 8)}
    return sorted(v for v in s if 0 <= v <= TOP)


def sizes():
    import dense_gemm_14_amd as g
    lib, n, count = g.load(), ctypes.c_size_t(0), 0

    def ask(name, *args):
        nonlocal count
        status = getattr(lib, name + "_workspace_size")(*args, ctypes.byref(n))
        assert status in (g.OK, g.ERR_UNSUPPORTED), (name, args, status)
        count += 1
    for rows in near(800):
        for cols in near(512, 8192, 16384):
            ask("gemm355_layer_norm_bwd", rows, cols)
    for tokens in near(1024, 3 << 15)[::3]:
        for vocab in near(1 << 20)[::3]:
            for cols in (0, 8, 520, 4096, 16384, TOP - 7):
                ask("gemm355_embedding_bwd", tokens, vocab, cols)
    for M in near(64)[::4]:
        for V in near(7680, 10240)[::4]:
            for K in (0, 8, 72, 1024, 4096, TOP - 7):
                ask("gemm_bf16_nt_cross_entropy", M, V, K)
                ask("gemm_bf16_nt_cross_entropy_bwd", M, V, K)
    print("sizes", count)


def launches(seed, count):
    from tests import test_dense_launches, test_ends_launches
    for t in (test_ends_launches, test_dense_launches):
        t.run(sys.argv[2], int(seed), int(count))
    # no tokens, and none of their arrays, over several pieces of the vocabulary
    rec = test_ends_launches.Recorder(sys.argv[2])
    rec.call("gemm_bf16_nt_cross_entropy_bwd", (0, 1 << 25, 64),
             lambda w, n: (0, 1 << 25, 64, None, None, 0, None, None, None, None, rec.DB, w, n, None))
    print("launches", sum(rec.seen.values()))


def test_size_queries(built):
    assert int(child("sizes", *built)[-1]) > 50000


def test_launches(built):
    assert int(child("launches", *built, "5", "300")[-1]) >= 4


if __name__ == "__main__":
    import dense_gemm_14_amd
    stand_in = ctypes.CDLL(sys.argv[2], ctypes.RTLD_GLOBAL)
    dense_gemm_14_amd.LIB_PATH = sys.argv[3]
    {"sizes": sizes, "launches": launches}[sys.argv[1]](*sys.argv[4:])
