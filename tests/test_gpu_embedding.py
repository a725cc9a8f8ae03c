"""Embedding and its gradient against 64-bit references on the GPU: every type,
odd numbers of tokens and ids, ids that are left out, ids that repeat up to all of
them, the table's gradient in place, repeatability."""
import pytest
import torch

import dense_gemm_14_amd as g
from tests.dense_util import close
from tests.gpu_util import need_gpu
from tests.rows_util import Array, embed, embed_bwd, randn

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def gen_of(seed):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return gen


def ids_of(gen, tokens, vocab, how, dtype=torch.int64):
    """how: 'any' (uniform, some left out), 'frequent' (the k-th about 1 / k as
    often as the first), 'one' (all the same), 'none' (all left out)."""
    if how == "none":
        ids = torch.where(torch.rand(tokens, generator=gen) < 0.5, -1, vocab)
    elif how == "one":
        ids = torch.full((tokens,), vocab // 2)
    elif how == "frequent":
        ids = (torch.exp(torch.rand(tokens, generator=gen, dtype=torch.float64) *
                         torch.log(torch.tensor(vocab + 1.0, dtype=torch.float64))).long() - 1).clamp(0, max(vocab - 1, 0))
    else:
        ids = torch.randint(0, max(vocab, 1), (tokens,), generator=gen)
        ids[torch.rand(tokens, generator=gen) < 0.2] = -100
        ids[torch.rand(tokens, generator=gen) < 0.1] = vocab
        if dtype == torch.int64:      # low words that are ids of the table
            ids[torch.rand(tokens, generator=gen) < 0.1] = (1 << 32) + 1
            ids[torch.rand(tokens, generator=gen) < 0.1] = -(1 << 32)
    return ids.to(dtype)


@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 8), (1, 1000, 4096), (4, 33, 520), (77, 300, 16), (5, 7, 24),
                                               (1001, 517, 1032), (3001, 100, 2056), (20000, 64, 64)])
@pytest.mark.parametrize("e_type", [BF16, FP32])
@pytest.mark.parametrize("y_type", [BF16, FP32])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_lookup(tokens, vocab, cols, e_type, y_type, id_type):
    need_gpu()
    print("embed", tokens, vocab, cols, e_type, y_type, id_type, flush=True)
    gen = gen_of(tokens + vocab + cols)
    ids, E = ids_of(gen, tokens, vocab, "any", id_type), randn(gen, vocab, cols, dtype=e_type)
    Y = Array(tokens, cols, dtype=y_type)
    for scale in (1.0, 22.627417):
        g.embedding(tokens, vocab, cols, ids.cuda(), E.cuda(), Y.t, scale)
        torch.cuda.synchronize()
        close(Y.get(), *embed(ids, E, scale, vocab, y_type), "Y")


def test_lookup_keeps_infinities_and_an_empty_table():
    need_gpu()
    E = torch.full((3, 8), float("inf"), dtype=BF16)
    E[1] = float("nan")
    Y = Array(4, 8)
    ids = torch.tensor([0, -1, 1, 2])
    g.embedding(4, 3, 8, ids.cuda(), E.cuda(), Y.t, 2.0)
    torch.cuda.synchronize()
    got = Y.get()
    assert got[0].isinf().all() and (got[1] == 0).all() and got[2].isnan().all() and got[3].isinf().all()
    g.embedding(4, 0, 8, ids.cuda(), None, Y.t, 2.0)
    torch.cuda.synchronize()
    assert (Y.get() == 0).all()


SIZES = [(1, 1, 8), (3, 1000, 520), (33, 7, 24), (64, 129, 4096), (777, 5001, 1000), (1024, 640, 520), (1025, 640, 520),
         (5000, 300, 136), (2050, 3, 1032), (9000, 70001, 72), (33000, 130001, 24),
         (98303, 1, 8), (98304, 1, 8), (99000, 50, 40), (102401, 2048, 24), (140001, 2049, 40), (99000, 130001, 16),
         (99000, 1048576, 8), (99000, 1048577, 8)]


def run_bwd(tokens, vocab, cols, ids, dY, R, scale, e_type, in_place=False):
    dE = Array(vocab, cols, dtype=e_type, fill=R if in_place else None)
    nb = g.embedding_bwd_workspace_size(tokens, vocab, cols)
    ws = torch.full((nb + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    r = None if R is None else dE.t if in_place else R.cuda()
    g.embedding_bwd(tokens, vocab, cols, ids.cuda(), dY.cuda(), r, dE.t, scale, ws, nb)
    torch.cuda.synchronize()
    assert (ws[nb:] == 0xFF).all(), "write past the workspace"
    return dE.get()


@pytest.mark.parametrize("tokens,vocab,cols", SIZES)
@pytest.mark.parametrize("how", ["any", "frequent", "one", "none"])
def test_gradient(tokens, vocab, cols, how):
    need_gpu()
    gen = gen_of(tokens + vocab + cols)
    for y_type, e_type, id_type, base in ((BF16, BF16, torch.int64, None), (FP32, BF16, torch.int32, "apart"),
                                          (BF16, FP32, torch.int64, "in place"), (FP32, FP32, torch.int32, "in place")):
        print("embed_bwd", tokens, vocab, cols, how, y_type, e_type, id_type, base, flush=True)
        ids = ids_of(gen, tokens, vocab, how, id_type)
        dY = randn(gen, tokens, cols, dtype=y_type)
        R = randn(gen, vocab, cols, dtype=e_type) if base else None
        got = run_bwd(tokens, vocab, cols, ids, dY, R, 3.25, e_type, base == "in place")
        close(got, *embed_bwd(ids, dY, R, 3.25, vocab, e_type), "dE")


def test_gradient_of_no_tokens():
    need_gpu()
    for R in (None, randn(gen_of(1), 50, 72)):
        got = run_bwd(0, 50, 72, torch.zeros(0, dtype=torch.int64), torch.zeros(0, 72, dtype=BF16), R, 2.0, BF16)
        assert torch.equal(got, torch.zeros(50, 72).double() if R is None else R.double())


def test_gradient_ignores_rows_that_are_left_out():
    # NaN in the rows of dY whose id is left out, and in the rows of R that no
    # token has: the first do not appear, the second stay
    need_gpu()
    gen = gen_of(5)
    ids = ids_of(gen, 500, 40, "any")
    dY, R = randn(gen, 500, 72), randn(gen, 40, 72)
    left = (ids < 0) | (ids >= 40)
    assert left.any()
    dY[left] = float("nan")
    ids[ids == 7] = 8
    R[7] = float("nan")
    got = run_bwd(500, 40, 72, ids, dY, R, 1.0, BF16)
    assert got[7].isnan().all()
    want, bound = embed_bwd(ids, torch.where(left[:, None], 0, dY), torch.nan_to_num(R), 1.0, 40, BF16)
    rest = torch.arange(40) != 7
    close(got[rest], want[rest], bound[rest], "dE")


@pytest.mark.parametrize("tokens,vocab,cols", [(6000, 500, 264), (100000, 5000, 24)])
def test_gradient_is_the_same_every_time(tokens, vocab, cols):
    need_gpu()
    gen = gen_of(6)
    ids, dY = ids_of(gen, tokens, vocab, "frequent"), randn(gen, tokens, cols, dtype=FP32)
    first = run_bwd(tokens, vocab, cols, ids, dY, None, 1.5, FP32)
    for _ in range(5):
        assert torch.equal(run_bwd(tokens, vocab, cols, ids, dY, None, 1.5, FP32), first)


def test_gradient_against_differences():
    # sum of W * Y over the lookup, changed in one element of the table at a time
    need_gpu()
    gen = gen_of(7)
    tokens, vocab, cols = 60, 9, 16
    ids = ids_of(gen, tokens, vocab, "any", torch.int32)
    E = torch.randint(-4, 5, (vocab, cols), generator=gen).float()
    W = torch.randint(-4, 5, (tokens, cols), generator=gen).float()
    got = run_bwd(tokens, vocab, cols, ids, W, None, 2.0, FP32)

    def total(table):
        Y = torch.empty(tokens, cols, device="cuda")
        g.embedding(tokens, vocab, cols, ids.cuda(), table.cuda(), Y, 2.0)
        return (Y.cpu().double() * W.double()).sum()
    for v in range(vocab):
        for c in (0, 7, 15):
            up, down = E.clone(), E.clone()
            up[v, c] += 1
            down[v, c] -= 1
            assert (total(up) - total(down)) / 2 == got[v, c]      # whole numbers: exact


def test_far_offsets():
    # a table of 4.3e9 elements' bytes and rows behind 2^32 bytes
    need_gpu()
    vocab, cols, tokens = 270000, 8192, 40
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    E = torch.zeros(vocab, cols, dtype=BF16, device="cuda")
    rows = torch.tensor([0, 131071, 131072, 262143, 262144, 262145, 269999], device="cuda")
    E[rows] = torch.randn(len(rows), cols, generator=gen, device="cuda").bfloat16()
    ids = rows[torch.randint(0, len(rows), (tokens,), generator=gen, device="cuda")]
    Y = torch.empty(tokens, cols, dtype=BF16, device="cuda")
    g.embedding(tokens, vocab, cols, ids, E, Y, 1.0)
    assert torch.equal(Y, E[ids])
    want = torch.zeros(len(rows), cols, dtype=torch.float64, device="cuda")
    whole = torch.randint(-3, 4, (tokens, cols), generator=gen, device="cuda").bfloat16()
    for i, r in enumerate(rows.tolist()):
        want[i] = whole[ids == r].double().sum(0)
    ws = torch.empty(g.embedding_bwd_workspace_size(tokens, vocab, cols), dtype=torch.uint8, device="cuda")
    E.fill_(float("nan"))
    g.embedding_bwd(tokens, vocab, cols, ids, whole, None, E, 1.0, ws)
    torch.cuda.synchronize()
    assert torch.equal(E[rows].double(), want)
    E[rows] = 0
    assert not E.any()
