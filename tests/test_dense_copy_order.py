"""The copy, wait, barrier and read order of the layer kernels' LDS rings, on the
host-side model of test_copy_order_model.py (a wave's copies complete in the
order it issued them; nothing else is assumed): the 256 x 256 kernel over work
items of different lengths, with and without reading an item's first fragments
again behind the epilogue, the 128 x 128 kernel's ring, and the small tiles',
which each wave keeps for itself."""
import os
import re

import pytest

from tests.test_copy_order_model import CSRC, Wave, _fails_with_looser_waits


def _src(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


# ---- 256 x 256 ------------------------------------------------------------------

COPIES, SLOTS, MIN_STEPS = 8, 5, 4


def test_large_constants_match_the_kernel():
    s = _src("dense_large.hpp")
    assert "constexpr int BIG_SLOTS = %d;" % SLOTS in s
    assert "COPIES = BLOCKS," in s and "bool TAIL, int BLOCKS = %d>" % COPIES in s
    assert re.search(r"constexpr int BIG_MIN_STEPS = %d;" % MIN_STEPS, s)
    assert re.search(r"if constexpr \(!first\)\s*wait_copies_le<COPIES>\(\);\s*lds_barrier\(\);", s)
    assert "mma2_copies(q, 0, Int<(q - a0) / d>{}, ring[4], a_off, tail);" in s
    assert "mma2_copies(q, 1, Int<(q - b0) / d>{}, ring[0], b_off, tail);" in s
    assert "read_a(ring[2], i);" in s and "read_b(ring[3], j);" in s
    assert "read_a(ring[0], i);" in s and "read_b(ring[1], BLOCKS - 1);" in s
    assert "read_a(ring[0], j);" in s and "read_b(ring[1], j);" in s      # read_first
    # an item: its first step, those in between, the last two; then every copy, the epilogue, the reads again
    assert re.search(r"step\(item.first \+ 2, Int<1>\{\}, Int<0>\{\}\);\s*for \(int s = 1; s < item.steps - 2; \+\+s\)", s)
    assert re.search(r"for \(int s = 0; s < 2; \+\+s\)\s*step\(after \+ s, Int<0>\{\}, Int<1>\{\}\);", s)
    assert s.index("step(after + s") < s.index("wait_all_copies();\n\n        const int ln") < s.index("if constexpr (REREAD)\n            read_first();")
    assert re.search(r"ring\[0\] = ring\[2\];\s*ring\[1\] = ring\[3\];\s*ring\[2\] = ring\[4\];\s*"
                     r"ring\[3\] = r0;\s*ring\[4\] = r1;", s)


def large_run(items, reread, blocks=COPIES):
    w, copies = Wave(SLOTS), blocks
    A, B = (lambda t, k: ("A", t, k)), (lambda t, k: ("B", t, k))
    ring = list(range(SLOTS))

    def first(t):
        for j in range(blocks - 1):
            if j < blocks // 2:
                w.read(A(t, 0), ring[0])
            w.read(B(t, 0), ring[1])
    for u, unit in enumerate((A(0, 0), B(0, 0), A(0, 1), B(0, 1))):
        w.copy(unit, u, copies)
    w.wait(0)
    w.barrier()
    first(0)
    for t, n in enumerate(items):
        for s in range(n):
            kt, ks = (t, s + 2) if s + 2 < n else (t + 1, s + 2 - n)
            nt, nx = (t, s + 1) if s + 1 < n else (t + 1, 0)
            w.copy(A(kt, ks), ring[4], copies)
            w.read(B(t, s), ring[1])
            for _ in range(blocks // 2):
                w.read(A(t, s), ring[0])
            w.wait_reads()
            if s:
                w.wait(copies)
            w.barrier()
            w.copy(B(kt, ks), ring[0], copies)
            for _ in range(blocks // 2):
                w.read(A(nt, nx), ring[2])
            for _ in range(blocks - 1):
                w.read(B(nt, nx), ring[3])
            ring = ring[2:] + ring[:2]
        w.wait(0)
        w.tick()            # the epilogue's stores: not ordered against copies
        if reread:
            first(t + 1)
    return w


@pytest.mark.parametrize("reread", [False, True])
@pytest.mark.parametrize("items", [[4], [4, 4, 4], [5, 9, 4], [40, 4, 17], [6, 6], [128, 9]])
@pytest.mark.parametrize("blocks", [8, 6])
def test_large_order(items, reread, blocks):
    large_run(items, reread, blocks)


@pytest.mark.parametrize("blocks", [8, 6])
def test_large_fragments_are_read_between_their_uses(blocks):
    # after the last pair that uses a fragment's registers, eight pairs before
    # the next that does; from a unit whose copies the middle of the step waits for
    s = _src("dense_large.hpp")
    half, rows = blocks * blocks // 2, blocks // 2
    for text in ("row(int q) { return (q < HALF ? 0 : ROWS) + q % ROWS; }", "col(int q) { return q % HALF / ROWS; }",
                 "BLOCKS == 8 ? (i < 4 ? 34 + 4 * i : 8 + 6 * (i - 4)) : i < 3 ? 19 + 3 * i : 5 + 3 * (i - 3);",
                 "BLOCKS == 8 ? 36 + 4 * j : 21 + 3 * j; }", "LAST_B_READ = 2;",
                 "return BLOCKS * c + 2; }", "return HALF + (last ? 2 : BLOCKS) * c; }"):
        assert text in s, text
    pairs = 2 * half
    uses = [((0 if q < half else rows) + q % rows, q % half // rows) for q in range(pairs)]
    assert sorted(uses) == [(i, j) for i in range(blocks) for j in range(blocks)]
    a_read = [(34 + 4 * i if i < 4 else 8 + 6 * (i - 4)) if blocks == 8 else (19 + 3 * i if i < 3 else 5 + 3 * (i - 3))
              for i in range(blocks)]
    b_read = [36 + 4 * j if blocks == 8 else 21 + 3 * j for j in range(blocks - 1)] + [2]
    for at, which in [(a, ("A", i)) for i, a in enumerate(a_read)] + [(b, ("B", j)) for j, b in enumerate(b_read)]:
        used = [q for q, (i, j) in enumerate(uses) if which in (("A", i), ("B", j))]
        if at >= half:     # the next step's
            assert max(used) <= at < pairs and min(used) + pairs - at >= 8
        else:              # this step's
            assert min(used) - at >= 8 and max(used) - pairs <= at
    for last in (False, True):     # every copy has its pair, in the half that may overwrite the slot
        assert 2 + blocks * (blocks // 2 - 1) < half and (2 if last else blocks) * (blocks // 2 - 1) < half


def test_large_model_catches_a_looser_wait():
    _fails_with_looser_waits(lambda nk, tiles: large_run([nk] * tiles, True), 8)
    _fails_with_looser_waits(lambda nk, tiles: large_run([nk] * tiles, True, 6), 8)


# ---- 128 x 128 -------------------------------------------------------------------

TILE_STAGES, TILE_COPIES = 4, 4


def test_tile_constants_match_the_kernel():
    s = _src("dense_tile.hpp")
    assert "constexpr int TILE_STAGES = %d;" % TILE_STAGES in s
    assert "constexpr int TILE_COPIES = %d;" % TILE_COPIES in s
    body = s[s.index("auto step = [&](int s, auto buf_c) {"):]
    order = ["copies(s + TILE_STAGES - 1);", "wait_reads();", "wait_copies_le<TILE_COPIES * (TILE_STAGES - 2)>();",
             "lds_barrier();", "oa.read(next"]
    at = [body.index(o) for o in order]
    assert at == sorted(at)


def tile_run(steps, _tiles=1):
    w = Wave(TILE_STAGES)
    for s in range(TILE_STAGES - 1):
        w.copy(s, s, TILE_COPIES)
    w.wait(TILE_COPIES * (TILE_STAGES - 2))
    w.barrier()
    w.read(0, 0)
    for s in range(steps):
        new = s + TILE_STAGES - 1
        w.copy(new, new % TILE_STAGES, TILE_COPIES)
        w.wait_reads()
        w.wait(TILE_COPIES * (TILE_STAGES - 2))
        w.barrier()
        for _ in range(8):
            w.read(s + 1, (s + 1) % TILE_STAGES)
    w.wait_reads()
    w.wait(0)
    assert w.proven == len(w.copies)      # none writes the LDS that the exchange uses


@pytest.mark.parametrize("steps", range(1, 20))
def test_tile_order(steps):
    tile_run(steps)


def test_tile_model_catches_a_looser_wait():
    _fails_with_looser_waits(tile_run, 8)


# ---- small tiles ------------------------------------------------------------------

def stages_of(mb, nb):
    return 20480 // ((mb + nb) * 2048)


def test_small_constants_match_the_kernel():
    s = _src("dense_small.hpp")
    assert "constexpr int small_stage(int mb, int nb) { return (mb + nb) * 2048; }" in s
    assert "constexpr int small_stages(int mb, int nb) { return 20480 / small_stage(mb, nb); }" in s
    body = s[s.index("for (int s = 0; s < slices; ++s) {"):]
    order = ["wait_copies_le<SLICE_COPIES * (STAGES - 1)>();", "oa.read(slot", "ob.read(slot", "wait_reads();",
             "copies(s + STAGES, slot);", "wait_all_copies();", "__syncthreads();"]
    at = [body.index(o) for o in order]
    assert at == sorted(at)


@pytest.mark.parametrize("mb,nb", [(1, 1), (1, 2), (1, 4), (2, 1), (2, 2), (4, 4)])
def test_small_order(mb, nb):
    stages, per = stages_of(mb, nb), 2 * (mb + nb)
    assert stages >= 1 and 8 * stages * (mb + nb) * 2048 <= 163840
    for slices in range(1, 12):
        issued, proven, slot_of = [], 0, {}
        for s in range(stages):
            issued += [s] * per
            slot_of[s] = s
        for s in range(slices):
            bound = per * (stages - 1)
            assert bound <= 63
            proven = max(proven, len(issued) - bound)
            assert all(u != s for u in issued[proven:]) and s in issued[:proven]     # the slice has landed
            # its reads are waited for before its stage is filled again
            slot_of[s + stages] = slot_of[s]
            issued += [s + stages] * per
