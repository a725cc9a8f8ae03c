"""Newton-Schulz where the guard of the division outweighs the norm: X then
starts at a small share r = |G| / (|G| + eps) of an orthogonal matrix's size and
has to keep its bits while the steps grow it."""
import math

import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_dense import gen_of, ortho_exact, run_ortho

pytestmark = pytest.mark.gpu
COEF = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("shape", [(2, 64, 64), (1, 256, 1032), (1, 1032, 256), (1, 520, 512), (1, 2056, 1032)])
@pytest.mark.parametrize("share", [1e-2, 1e-4, None], ids=["1e-2", "1e-4", "limit"])
def test_norm_far_below_eps(shape, share):
    need_gpu()
    gen = gen_of(*shape, 101)
    G = torch.randn(*shape, generator=gen).float()
    G /= G.double().flatten(1).norm(dim=1)[:, None, None].float()      # norms of about 1
    r = share or 2.0 ** -26 * math.sqrt(shape[1] * shape[2])
    eps = torch.tensor(1.0 / r - 1.0).float().item()
    print("share", shape, r, flush=True)
    got, want = run_ortho(G, 5, COEF, eps), ortho_exact(G, 5, COEF, eps)
    rel = ((got - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max().item()
    # as in test_newton_schulz: three roundings to FP16 in each of five steps,
    # which at the limit are those of FP16's smallest normal values still, and
    # the BF16 rounding of the result
    assert rel <= 15 ** 0.5 * 2.0 ** -11 * 2 + 2.0 ** -8 / 3 ** 0.5, rel
