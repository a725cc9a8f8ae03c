"""The workspaces of the embedding, layer norm and cross entropy calls: the size that a
call's query gives is taken, one byte less is refused before anything is launched; and
the widest rows that an int holds. In a process of its own, against the stand-in for the
HIP runtime."""
import os
import random
import subprocess
import sys

import pytest

import dense_gemm_14_amd as g
from tests.test_ends_launches import Recorder, log_size

HERE = os.path.dirname(os.path.abspath(__file__))
WIDEST = (1 << 31) - 8


class Strict(Recorder):
    refused = 0

    def launched(self, status, what):
        """Whether the call was taken; a refused one has launched nothing."""
        if status == g.OK:
            self.take(status, what)
            return True
        assert status == g.ERR_UNSUPPORTED, (what, status)
        assert self.shim.recorder_take() == 0, what
        self.refused += 1
        return False

    def call(self, name, sizes, args):
        nb, fn = self.size(name, *sizes), getattr(self.lib, name)
        if nb > 0:
            assert not self.launched(fn(*args(self.WS, nb - 1)), (name, sizes, nb - 1)), (name, sizes)
            assert not self.launched(fn(*args(None, 0)), (name, sizes, 0)) if name.startswith("gemm355") else True
        assert self.launched(fn(*args(self.WS if nb else None, nb)), (name, sizes, nb)), (name, sizes)

    def norm_bwd(self, M, N, wanted):
        """The query's size is that of the type of X that takes more."""
        name, nb = "gemm355_layer_norm_bwd", self.size("gemm355_layer_norm_bwd", M, N)
        outs = [p if on else None for p, on in zip((self.E, self.DG, self.DB), wanted)]
        for short in (0, 1):
            if nb == 0 and short:
                continue
            taken = [self.launched(self.lib.gemm355_layer_norm_bwd(
                M, N, xt, self.X, 1, self.GAMMA, self.MEAN, self.RSTD, self.Y, self.R, *outs, self.WS if nb else None,
                nb - short, None), (name, M, N, xt, short)) for xt in (0, 1)]
            assert all(taken) if not short else not all(taken), (M, N, nb, short, taken)


def run(shim, seed, count):
    rng, rec = random.Random(seed), Strict(shim)
    for M, N in ((1, WIDEST), (300, WIDEST), (1, 1 << 22), (900, 8200), (900, 16384), (900, 16392), (1 << 20, 8192)):
        rec.norm_bwd(M, N, (1, 1, 1))
        assert rec.launched(rec.lib.gemm355_layer_norm(M, N, 0, rec.X, 0, None, None, 1e-5, rec.Y, None, None, None), (M, N))
    for T, V in ((1, 2), (4, 300), (1024, 1), (1025, 40)):
        rec.embedding(T, V, WIDEST // (1 if T < 100 else 4) // 8 * 8, rng)
    for _ in range(count):
        rec.embedding(log_size(rng, 1, 1000000), log_size(rng, 1, 300000), log_size(rng, 8, 16384, 8), rng)
        rec.norm_bwd(log_size(rng, 1, 20000), log_size(rng, 8, 40000, 8), rng.choice([(1, 1, 1), (1, 0, 0), (0, 1, 0), (1, 0, 1)]))
        rec.lib.gemm355_force_layer_kernel(rng.choice([0, 0, 0, 1, 2, 3, 4, 5]))
        rec.entropy(log_size(rng, 1, 20000), log_size(rng, 1, 300000), log_size(rng, 8, 8192, 8), rng)
        # around the vocabularies up to which small gradients are summed in another way
        rec.entropy(log_size(rng, 1, 400), rng.randrange(7000, 11000), log_size(rng, 8, 2048, 8), rng)
        rec.lib.gemm355_force_layer_kernel(0)
    print("refused", rec.refused)


@pytest.mark.parametrize("seed", [1, 2])
def test_one_byte_less_is_refused(seed, tmp_path):
    g.load()     # built here if nothing is
    out = str(tmp_path / "recorder.so")
    subprocess.run(["gcc", "-O1", "-Wall", "-shared", "-fPIC", "-o", out, os.path.join(HERE, "launch_recorder.c")], check=True)
    p = subprocess.run([sys.executable, "-m", "tests.test_ends_workspaces", out, str(seed), "200"],
                       cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-3000:]
    assert int(p.stdout.split()[-1]) > 500


if __name__ == "__main__":
    run(sys.argv[1], int(sys.argv[2]), int(sys.argv[3]))
