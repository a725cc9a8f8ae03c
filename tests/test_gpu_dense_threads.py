"""Layer calls from several threads at once, each on its own stream, by themselves
and while another thread changes the kernels' override. Every result is compared
inside its thread with the one right value that sums of whole numbers have,
whichever kernel ran, and a thread's error is the test's."""
import threading

import pytest
import torch

import dense_gemm_14_amd as g
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


class Block:
    """A gated layer and a linear one with their gradients, on whole numbers."""

    def __init__(self, M, N, K, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        whole = lambda *s: torch.randint(-1, 2, s, generator=gen, device="cuda").to(torch.bfloat16)
        new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
        self.A, self.B, self.R, self.dC = whole(M, K), whole(2 * N, K), whole(M, 2 * N), whole(M, N)
        self.ws = torch.empty(max(g.gated_workspace_size(M, N, K), g.gated_bwd_workspace_size(M, N, K),
                                  g.bias_act_res_workspace_size(M, 2 * N, K),
                                  g.bias_act_bwd_workspace_size(M, 2 * N, K, g.ACT_NONE), 1 << 20), dtype=torch.uint8,
                              device="cuda")
        self.Z, self.C, self.Y = new(M, 2 * N), new(M, N), new(M, 2 * N)
        self.dA, self.dB, self.db = new(M, K), new(2 * N, K), new(2 * N)
        self.lA, self.lB, self.lb = new(M, K), new(2 * N, K), new(2 * N)
        a, b, d, r = (x.float() for x in (self.A, self.B, self.dC, self.R))
        z = a @ b.t()
        self.Zin = z.clamp(-8, 8).to(torch.bfloat16)     # pre-activations for the backward call, exact in BF16
        zi = self.Zin.float()
        dz = torch.cat([d * zi[:, N:] * (zi[:, :N] > 0), d * zi[:, :N].clamp(min=0)], 1)
        bf = lambda t: t.to(torch.bfloat16)
        self.calls = [
            (lambda: g.gemm_bf16_nt_gated(M, N, K, self.A, self.B, None, g.ACT_RELU, self.Z, self.C, self.ws),
             [(self.Z, bf(z)), (self.C, bf(z[:, :N].clamp(min=0) * z[:, N:]))]),
            (lambda: g.gemm_bf16_nt_bias_act_res(M, 2 * N, K, self.A, self.B, None, g.ACT_RELU, self.R, None, self.Y, self.ws),
             [(self.Y, bf(z.clamp(min=0) + r))]),
            (lambda: g.gemm_bf16_nt_gated_bwd(M, N, K, self.A, self.B, self.Zin, g.ACT_RELU, self.dC, self.dA, self.dB,
                                              self.db, self.ws),
             [(self.dA, bf(dz @ b)), (self.dB, bf(dz.t().contiguous() @ a)), (self.db, bf(dz.sum(0)))]),
            (lambda: g.gemm_bf16_nt_bias_act_bwd(M, 2 * N, K, self.A, self.B, None, g.ACT_NONE, self.R, self.lA, self.lB,
                                                 self.lb, self.ws),
             [(self.lA, bf(r @ b)), (self.lB, bf(r.t().contiguous() @ a)), (self.lb, bf(r.sum(0)))])]
        self.ran = 0

    def round(self, may_refuse):
        """Every call once, its outputs checked; counts the calls that ran."""
        for i, (call, outputs) in enumerate(self.calls):
            for out, _ in outputs:
                out.view(torch.int16).fill_(0x7FC1)
            try:
                call()
            except g.Gemm355Error as e:
                assert may_refuse and e.status == g.ERR_UNSUPPORTED, e
                continue
            torch.cuda.current_stream().synchronize()
            for k, (out, want) in enumerate(outputs):
                assert torch.equal(out, want), (i, k, int((out != want).sum()))
            self.ran += 1


def in_threads(works):
    """Runs the functions in a thread each and raises the first error of any."""
    errors = []

    def guarded(work):
        try:
            work()
        except BaseException as e:      # a thread's error does not end the test by itself
            errors.append(e)
    threads = [threading.Thread(target=guarded, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("toggled", [False, True], ids=["alone", "toggled"])
def test_every_call_of_every_thread_is_right(toggled):
    need_gpu()
    blocks = [Block(130 + 70 * i, 264, 520, 90 + i) for i in range(4)]
    for b in blocks:
        b.round(False)
        b.ran = 0
    torch.cuda.synchronize()
    done = threading.Event()
    left = [len(blocks)]
    lock = threading.Lock()

    def work(b):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(12):
                    b.round(toggled)
        finally:
            with lock:
                left[0] -= 1
                if left[0] == 0:
                    done.set()

    def toggle():
        kernels = [g.LAYER_LARGE, g.LAYER_SPLIT, g.LAYER_TILE, g.LAYER_SMALL, g.LAYER_NARROW, g.LAYER_AUTO]
        i = 0
        while not done.wait(1e-4):
            g.force_layer_kernel(kernels[i % len(kernels)])
            i += 1
    print("threads", toggled, flush=True)
    try:
        in_threads([lambda b=b: work(b) for b in blocks] + ([toggle] if toggled else []))
    finally:
        g.force_layer_kernel(g.LAYER_AUTO)
    torch.cuda.synchronize()
    for b in blocks:
        assert b.ran == 48 if not toggled else b.ran >= 12, b.ran
