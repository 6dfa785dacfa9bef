"""CPU model check of the attention-weight kernel's mbarrier pipeline (weights_protocol_model.py):
pieces of every small shape in a row, both ring lengths of its K stages, many random interleavings;
planted errors must fail, and every role must leave when a wait times out."""

import random

import pytest

from weights_protocol_model import weights

STAGES = pytest.mark.parametrize("S", [4, 8], ids=["d128", "d64"])


@STAGES
def test_single_pieces(S):
    weights([], S, 0)
    for n in range(1, 11):
        for jobs in range(1, 5):
            for seed in range(4):
                weights([(n, jobs)], S, seed)


@STAGES
def test_pieces_in_a_row(S):
    rng = random.Random(3)
    for k in range(80):
        weights([(rng.randint(1, 5), rng.randint(1, 3)) for _ in range(rng.randint(0, 9))], S, k)
        weights([(1, 1)] * rng.randint(5, 12), S, k)  # jobs of one tile: only one warpgroup works


@STAGES
def test_timeout_every_role_leaves(S):
    rng = random.Random(5)
    for k in range(10):
        pieces = [(rng.randint(1, 5), rng.randint(1, 3)) for _ in range(5)]
        spins = weights(pieces, S, k).spins
        for at in sorted(rng.sample(range(1, max(2, spins + 1)), min(8, spins))):
            sim = weights(pieces, S, k, abort_at=at)
            assert sim.abort and sim.exit_ops == 0 and sim.exit_copies == 0


@pytest.mark.parametrize("bug", ["mma_no_s_wait", "no_q_wait", "early_k_release", "early_piece_release",
                                 "three places for statistics"])
def test_checker_catches_planted_errors(bug):
    rng = random.Random(7)
    for seed in range(400):
        pieces = [(rng.choice([1, 1, 2, 6]), rng.choice([1, 1, 2])) for _ in range(10)]
        try:
            if bug.startswith("three"):
                weights(pieces, 4, seed, stats=3)
            else:
                weights(pieces, 2 if bug == "early_k_release" else 4, seed, bug=bug)
        except AssertionError:
            return
    raise AssertionError("not caught")
