"""CPU model check of the paged tensor-core kernel's mbarrier pipeline (paged_protocol_model.py):
pieces of every small shape in a row, both ring lengths of its K and V stages, one or both tile
slots, many random interleavings; planted errors must fail, and every role must leave when a wait
times out."""

import random

import pytest

from paged_protocol_model import paged

SHAPES = pytest.mark.parametrize("twin,S", [(False, 2), (False, 4), (True, 2), (True, 4)],
                                 ids=["two tiles d128", "two tiles d64", "one tile d128", "one tile d64"])


def _pieces(rng, twin, count, most):
    if twin:
        return [rng.randint(0, most) for _ in range(count)]
    out = []
    for _ in range(count):  # tile 1's rows come after tile 0's: as many key tiles, or more, or none
        n0 = rng.randint(0, most)
        out.append((n0, rng.choice([0, n0, min(most, n0 + 1)]) if n0 else 0))
    return out


@SHAPES
def test_single_pieces(twin, S):
    shapes = range(10) if twin else [(a, b) for a in range(7) for b in range(7) if a or not b]
    for n in shapes:
        for seed in range(4):
            paged([n], S, seed, twin)


@pytest.mark.parametrize("S", [2, 4])
def test_first_query_tile_without_keys(S):
    """Rows of the first tile that see none of a piece's keys, next to a second tile that does."""
    rng = random.Random(9)
    for n in range(7):
        for seed in range(4):
            paged([(0, n)], S, seed, False)
    for k in range(60):
        pieces = [(rng.randint(0, 4), rng.randint(0, 4)) for _ in range(rng.randint(1, 9))]
        spins = paged(pieces, S, k, False).spins
        for at in sorted(rng.sample(range(1, max(2, spins + 1)), min(3, spins))):
            sim = paged(pieces, S, k, False, abort_at=at)
            assert sim.abort and sim.exit_ops == 0 and sim.exit_copies == 0


@SHAPES
def test_pieces_in_a_row(twin, S):
    rng = random.Random(3)
    for k in range(60):
        paged(_pieces(rng, twin, rng.randint(0, 9), 5), S, k, twin)


@SHAPES
def test_timeout_every_role_leaves(twin, S):
    rng = random.Random(5)
    for k in range(8):
        pieces = _pieces(rng, twin, 4, 5)
        spins = paged(pieces, S, k, twin).spins
        for at in sorted(rng.sample(range(1, max(2, spins + 1)), min(8, spins))):
            sim = paged(pieces, S, k, twin, abort_at=at)
            assert sim.abort and sim.exit_ops == 0 and sim.exit_copies == 0


@pytest.mark.parametrize("twin,bug", [(False, "mma_no_q_wait"), (True, "mma_no_q_wait"), (True, "twin_no_wait"),
                                      (False, "early_v_release"), (True, "early_v_release"),
                                      (False, "early_piece_release"), (True, "early_piece_release")])
def test_checker_catches_planted_errors(twin, bug):
    pieces = [5, 4, 7, 3, 2, 6] if twin else [(5, 5), (4, 0), (3, 4), (2, 2), (1, 1), (3, 3)]
    for seed in range(200):
        try:
            paged(pieces, 2, seed, twin, bug=bug)
        except AssertionError:
            return
    raise AssertionError("not caught")
