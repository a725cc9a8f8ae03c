"""The loss's gradients around the vocabularies from which on small products are summed
in another way (7680 ids: split 128 x 128 tiles; 10240: two launches instead of one),
against 64 bits, with the bounds of test_gpu_cross_entropy.py."""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_cross_entropy import backward_reference, check, forward_reference, inputs, run_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [7679, 7680, 7681, 9001, 10239, 10240, 10241, 12001])
@pytest.mark.parametrize("M,K,skip", [(2, 1032, 0.0), (33, 264, 0.5), (150, 88, 0.1), (300, 64, 0.9), (400, 520, 0.1)])
def test_gradients_between_the_limits(M, V, K, skip):
    need_gpu()
    print("ce sums", M, V, K, flush=True)
    A, B, t, w = (x.cuda() for x in inputs(M, V, K, skip=skip))
    lse = forward_reference(A, B, t)["lse"][0].float()
    want = backward_reference(A, B, t, lse, w)
    for wanted in (("dA", "dB"), ("dA",), ("dB",)):
        check(run_bwd(A, B, t, lse, w, wanted), want)
