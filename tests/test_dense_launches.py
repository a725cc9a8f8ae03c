"""Every launch of the layer calls has the threads that its kernel is compiled
for, and fewer than 2^32 work-items: the built library runs in a process of its
own against a stand-in for the HIP runtime (launch_recorder.c) that writes the
launches down, over sizes of the whole range, every choice of gradients and
every forced kernel."""
import ctypes
import os
import random
import re
import subprocess
import sys

import pytest

import dense_gemm_14_amd as g

HERE = os.path.dirname(os.path.abspath(__file__))

# threads of the kernels that have one number of them; the small-tile kernels'
# are 64 times the last of their template arguments
THREADS = {"dense_tile_kernel": 512, "dense_reduce_kernel": 256, "dense_large_kernel": 256,
           "dense_large_reduce_kernel": 256, "dense_grad_kernel": 256, "dense_bias_kernel": 512, "ns_norm_kernel": 256,
           "ns_scale_kernel": 256}
GRADIENTS = range(1, 8)      # bits: dA 1, dB 2, dbias 4
SUBSETS = {1: "dA", 2: "dB", 3: "dA dB", 4: "dbias", 5: "dA dbias", 6: "dB dbias", 7: "dA dB dbias"}


def kernel_of(mangled):
    """(name, threads it is compiled for) of a kernel's mangled name."""
    name = re.match(r"_ZN7gemm3555dense\d+([a-z_]+?_kernel)", mangled).group(1)
    if name in THREADS:
        return name, THREADS[name]
    assert name in ("dense_small_kernel", "dense_small_bwd_kernel"), mangled
    return name, 64 * int(re.search(r"Li(\d+)EEEv", mangled).group(1))


class Recorder:
    """The library on the stand-in; only in a process of its own."""

    def __init__(self, shim):
        self.shim = ctypes.CDLL(shim, ctypes.RTLD_GLOBAL)
        self.shim.recorder_name.restype = ctypes.c_char_p
        self.shim.recorder_blocks.restype = ctypes.c_uint
        self.lib = g.load()
        assert self.size("gemm_bf16_nt_workspace_size", 8, 8, 8) == 0
        self.seen = {}

    def size(self, name, *args):
        n = ctypes.c_size_t(0)
        assert getattr(self.lib, name)(*args, ctypes.byref(n)) == g.OK, (name, args)
        return n.value

    def check(self, status, what):
        count = self.shim.recorder_take()
        assert status == g.OK and count > 0, (what, status, count)
        for i in range(count):
            mangled = self.shim.recorder_name(i).decode()
            name, threads = kernel_of(mangled)
            have, blocks = self.shim.recorder_threads(i), self.shim.recorder_blocks(i)
            assert have == threads, "%s: %s launched with %d threads, compiled for %d" % (what, mangled, have, threads)
            assert 0 < blocks * have < 1 << 32, (what, mangled, blocks, have)
            self.seen[name, threads] = self.seen.get((name, threads), 0) + 1

    # addresses far apart, never read
    A, B, BIAS, R, Z, C, DC, DA, DB, DBIAS, WS = (i << 44 for i in range(1, 12))

    def forward(self, gated, M, N, K, act):
        call = "gemm_bf16_nt_gated" if gated else "gemm_bf16_nt_bias_act_res"
        nb = self.size(call + "_workspace_size", M, N, K)
        args = (M, N, K, self.A, self.B, self.BIAS, act, *(() if gated else (self.R,)), self.Z, self.C, self.WS, nb, None)
        self.check(getattr(self.lib, call)(*args), "%s %s" % (call, (M, N, K, act)))

    def backward(self, gated, M, N, K, act, wanted):
        call = "gemm_bf16_nt_gated_bwd" if gated else "gemm_bf16_nt_bias_act_bwd"
        nb = self.size(call + "_workspace_size", M, N, K, *(() if gated else (act,)))
        outs = [p if wanted >> i & 1 else None for i, p in enumerate((self.DA, self.DB, self.DBIAS))]
        status = getattr(self.lib, call)(M, N, K, self.A, self.B, self.Z, act, self.DC, *outs, self.WS, nb, None)
        self.check(status, "%s %s for %s" % (call, (M, N, K, act), SUBSETS[wanted]))

    def ortho(self, batch, rows, cols, fp32):
        nb = self.size("gemm355_newton_schulz_workspace_size", batch, rows, cols)
        status = self.lib.gemm355_newton_schulz(batch, rows, cols, int(fp32), self.A, 2, 3.0, -4.0, 2.0, 0.0, self.C,
                                                self.WS, nb, None)
        self.check(status, "newton_schulz %s" % ((batch, rows, cols, fp32),))


def log_size(rng, low, high, of):
    v = int(low * (high / low) ** rng.random())
    return max(low, v // of * of)


def run(shim, seed, count):
    rng, rec = random.Random(seed), Recorder(shim)
    fixed = [(1, 4096, 4096), (8, 4096, 4096), (64, 4096, 4096), (128, 4096, 4096), (64, 2048, 2048),
             (1310, 168, 6288), (1310, 6288, 168), (4096, 128, 4096), (301, 1384, 512), (8192, 1024, 1024)]
    sizes = fixed + [(log_size(rng, 1, 8192, 1), log_size(rng, 8, 8192, 8), log_size(rng, 8, 8192, 8))
                     for _ in range(count)]
    for M, N, K in sizes:
        rec.lib.gemm355_force_layer_kernel(rng.choice([0, 0, 0, 0, 1, 2, 3, 4, 4, 5]) if (M, N, K) not in fixed else 0)
        for gated in (False, True):
            act = rng.randrange(4)
            rec.forward(gated, M, N, K, act)
            for wanted in GRADIENTS:
                rec.backward(gated, M, N, K, act, wanted)
    # the most matrices of the largest size that the card holds: more elements
    # than one launch may have work-items
    for sizes in ((65535, 16, 32776), (65535, 32, 16384), (40000, 72, 11656)):
        rec.lib.gemm355_force_layer_kernel(0)
        rec.ortho(*sizes, False)
    for _ in range(count // 4):
        rec.lib.gemm355_force_layer_kernel(rng.choice([0, 0, 1, 2, 3, 4, 5]))
        rec.ortho(rng.choice([1, 2, 5, 12]), log_size(rng, 8, 4096, 8), log_size(rng, 8, 4096, 8), rng.random() < 0.5)
    # every kernel and every number of waves was among them
    for name, threads in [*THREADS.items(), *[("dense_small_kernel", 64 * w) for w in (1, 2, 4, 8)],
                          ("dense_small_bwd_kernel", 256), ("dense_small_bwd_kernel", 512)]:
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
    p = subprocess.run([sys.executable, "-m", "tests.test_dense_launches", recorder, str(seed), "600"],
                       cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-3000:]
    assert int(p.stdout.split()[-1]) > 10000


if __name__ == "__main__":
    run(sys.argv[1], int(sys.argv[2]), int(sys.argv[3]))
