"""Every launch of the embedding, layer norm and cross entropy calls has the threads
that its kernel is compiled for and fewer than 2^32 work-items, and its workspace
is the size that the call asks for: the built library in a process of its own
against a stand-in for the HIP runtime, over sizes of the whole range and the
largest ones."""
import ctypes
import os
import random
import re
import subprocess
import sys

import pytest

import dense_gemm_14_amd as g

HERE = os.path.dirname(os.path.abspath(__file__))
THREADS = {"embed_kernel": 256, "embed_order_kernel": 1024, "embed_sums_kernel": 256, "embed_few_kernel": 256,
           "embed_join_kernel": 512, "norm_kernel": 256, "norm_wide_kernel": 1024, "norm_bwd_kernel": 1024,
           "norm_sums_kernel": 1024, "embed_count_kernel": 1024, "embed_scan_kernel": 1024, "embed_place_kernel": 1024,
           "ce_prep_kernel": 256, "ce_join_kernel": 256, "dense_tile_kernel": 512,
           "dense_reduce_kernel": 256, "dense_reduce_many_kernel": 512, "dense_large_kernel": 256, "dense_large_reduce_kernel": 256}


def kernel_of(mangled):
    """(name, threads it is compiled for) of a kernel's mangled name."""
    name = re.match(r"_ZN7gemm355\d[a-z]+?\d+([a-z_]+?_kernel)", mangled).group(1)
    if name == "norm_bwd_direct_kernel":     # the last argument: eights of columns of a lane, 0 for very wide rows
        return name, 256 if int(re.search(r"Li(\d+)EEEv", mangled).group(1)) else 1024
    if name in ("dense_small_kernel", "dense_small_loss_kernel"):
        return name, 64 * int(re.search(r"Li(\d+)EEEv", mangled).group(1))
    return name, THREADS[name]


class Recorder:
    """The library on the stand-in; only in a process of its own."""

    IDS, E, R, Y, X, GAMMA, BETA, MEAN, RSTD, DG, DB, WS = (i << 45 for i in range(1, 13))

    def __init__(self, shim):
        self.shim = ctypes.CDLL(shim, ctypes.RTLD_GLOBAL)
        self.shim.recorder_name.restype = ctypes.c_char_p
        self.shim.recorder_blocks.restype = ctypes.c_uint
        self.lib = g.load()
        self.seen = {}

    def size(self, name, *args):
        n = ctypes.c_size_t(0)
        assert getattr(self.lib, name + "_workspace_size")(*args, ctypes.byref(n)) == g.OK, (name, args)
        return n.value

    def take(self, status, what):
        count = self.shim.recorder_take()
        assert status == g.OK and count > 0, (what, status, count)
        for i in range(count):
            mangled = self.shim.recorder_name(i).decode()
            name, threads = kernel_of(mangled)
            have, blocks = self.shim.recorder_threads(i), self.shim.recorder_blocks(i)
            assert have == threads, "%s: %s launched with %d threads, compiled for %d" % (what, mangled, have, threads)
            assert 0 < blocks * have < 1 << 32, (what, mangled, blocks, have)
            self.seen[name, threads] = self.seen.get((name, threads), 0) + 1

    def call(self, name, sizes, args):
        """args(workspace, its bytes) -> the call's arguments. One byte less is refused."""
        nb = self.size(name, *sizes)
        fn = getattr(self.lib, name)
        if nb > 0:
            assert fn(*args(self.WS, nb - 1)) in (g.ERR_UNSUPPORTED, g.OK), (name, sizes)
            self.shim.recorder_take()
        self.take(fn(*args(self.WS if nb else None, nb)), "%s %s" % (name, sizes))

    def embedding(self, T, V, K, rng):
        it, et, yt = rng.randrange(2), rng.randrange(2), rng.randrange(2)
        self.take(self.lib.gemm355_embedding(T, V, K, it, self.IDS, et, self.E, 2.0, yt, self.Y, None), "embedding %s" % ((T, V, K),))
        r = rng.choice([None, self.R, self.E])
        self.call("gemm355_embedding_bwd", (T, V, K),
                  lambda w, n: (T, V, K, it, self.IDS, yt, self.Y, 2.0, et, r, self.E, w, n, None))

    def norm(self, M, N, rng):
        xt, wt = rng.randrange(2), rng.randrange(2)
        self.take(self.lib.gemm355_layer_norm(M, N, xt, self.X, wt, self.GAMMA, self.BETA, 1e-5, self.Y, self.MEAN, self.RSTD,
                                              None), "layer_norm %s" % ((M, N),))
        wanted = rng.choice([(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 1, 1), (1, 0, 1)])
        outs = [p if on else None for p, on in zip((self.E, self.DG, self.DB), wanted)]
        self.call("gemm355_layer_norm_bwd", (M, N),
                  lambda w, n: (M, N, xt, self.X, wt, self.GAMMA, self.MEAN, self.RSTD, self.Y, self.R, *outs, w, n, None))

    def entropy(self, M, V, K, rng):
        it = rng.randrange(2)
        if M > 0:
            self.call("gemm_bf16_nt_cross_entropy", (M, V, K),
                      lambda w, n: (M, V, K, self.X, self.E, it, self.IDS, self.MEAN, self.RSTD, w, n, None))
        wanted = rng.choice([(1, 1), (1, 0), (0, 1)])
        outs = [p if on else None for p, on in zip((self.Y, self.DB), wanted)]
        if K > 0 and M <= 4000000 and ((M > 0 and wanted[0]) or (V > 0 and wanted[1])):
            self.call("gemm_bf16_nt_cross_entropy_bwd", (M, V, K),
                      lambda w, n: (M, V, K, self.X, self.E, it, self.IDS, self.RSTD, self.MEAN, *outs, w, n, None))


def log_size(rng, low, high, of=1):
    v = int(low * (high / low) ** rng.random())
    return max(low, v // of * of)


def run(shim, seed, count):
    rng, rec = random.Random(seed), Recorder(shim)
    # the largest: more rows and columns than one launch has threads for
    for T, V, K in ((2147483647, 1 << 30, 8), (100000000, 1 << 30, 512), (2147483647, 1, 8), (1, 1 << 30, 1024),
                    (1024, 1 << 30, 8), (1025, 300000, 65536), (0, 1000, 8)):
        if T > 0:
            rec.embedding(T, V, K, rng)
        else:
            rec.call("gemm355_embedding_bwd", (T, V, K),
                     lambda w, n: (T, V, K, 0, rec.IDS, 0, rec.Y, 2.0, 0, None, rec.E, w, n, None))
    for M, N in ((2147483647, 8), (2147483647, 512), (1, 1 << 30), (500, 1 << 31 - 9), (100000000, 4096), (1 << 20, 1 << 20)):
        rec.norm(M, N, rng)
    for M, V, K in ((1 << 18, 100000, 2048), (1, 1 << 27, 8), (1, 1000, 1 << 21), (100000, 200000, 512), (0, 100, 64),
                    (33, 0, 64), (4000000, 1000, 8), (260000, 300, 4096), (1 << 26, 100, 8), (1 << 26, 300, 0)):
        rec.entropy(M, V, K, rng)
    n = ctypes.c_size_t(7)
    for sizes in ((8000000, 1000, 8), (261500, 300, 4096)):
        assert rec.lib.gemm_bf16_nt_cross_entropy_bwd_workspace_size(*sizes, ctypes.byref(n)) == g.ERR_UNSUPPORTED, sizes
    # tiles of the logits beyond 32 bits: pieces
    rec.lib.gemm355_force_layer_kernel(5)
    args = (4000000, 1 << 20, 8)
    nb = rec.size("gemm_bf16_nt_cross_entropy", *args)
    assert nb > args[0] * args[1] // 16 and rec.lib.gemm_bf16_nt_cross_entropy(
        *args, rec.X, rec.E, 0, rec.IDS, rec.MEAN, rec.RSTD, 1 << 52, nb, None) == g.OK
    assert rec.shim.recorder_take() > 100
    rec.lib.gemm355_force_layer_kernel(0)
    for _ in range(count):
        rec.lib.gemm355_force_layer_kernel(0)
        rec.entropy(log_size(rng, 1, 3000), log_size(rng, 1, 3000), log_size(rng, 8, 2048, 8), rng)
        rec.embedding(log_size(rng, 1, 1000000), log_size(rng, 1, 300000), log_size(rng, 8, 16384, 8), rng)
        rec.norm(log_size(rng, 1, 20000), log_size(rng, 8, 40000, 8), rng)
        rec.lib.gemm355_force_layer_kernel(rng.choice([0, 0, 0, 1, 2, 3, 4, 5]))
        rec.entropy(log_size(rng, 1, 20000), log_size(rng, 1, 300000), log_size(rng, 8, 8192, 8), rng)
    rec.lib.gemm355_force_layer_kernel(0)
    for name, threads in [*THREADS.items(), ("norm_bwd_direct_kernel", 256), ("norm_bwd_direct_kernel", 1024),
                          *[("dense_small_kernel", 64 * w) for w in (1, 2, 4, 8)], ("dense_small_loss_kernel", 256),
                          ("dense_small_loss_kernel", 512)]:
        assert rec.seen.get((name, threads)), (name, threads, rec.seen)
    print("launches", sum(rec.seen.values()))


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("recorder") / "recorder.so")
    subprocess.run(["gcc", "-O1", "-Wall", "-shared", "-fPIC", "-o", out, os.path.join(HERE, "launch_recorder.c")],
                   check=True)
    return out


@pytest.mark.parametrize("seed", [1, 2])
def test_launches_have_their_kernels_threads(recorder, seed):
    g.load()     # built here if nothing is
    p = subprocess.run([sys.executable, "-m", "tests.test_ends_launches", recorder, str(seed), "300"],
                       cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-3000:]
    assert int(p.stdout.split()[-1]) > 3000


if __name__ == "__main__":
    run(sys.argv[1], int(sys.argv[2]), int(sys.argv[3]))
