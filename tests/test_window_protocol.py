"""The barriers of window_attn's kernel on pairs of SMs in random orders of its roles (no GPU)."""

from __future__ import annotations

import random

import pytest

from tests import _window_protocol as protocol

BLOCKS = [[1], [1, 1, 1, 2, 3], [0, 1, 2, 3, 4, 5], [1, 1, 2, 5, 9], list(range(14))]


@pytest.fixture(scope="module")
def source():
    return protocol.Source()


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("seed", range(20))
def test_no_wait_is_early_late_or_endless(source, codes, seed):
    rng = random.Random(seed)
    for i in range(2):
        blocks = BLOCKS[(seed + i) % len(BLOCKS)]
        protocol.Pair(source, codes, [rng.choice(blocks) for _ in range(rng.randrange(4, 25))], rng).run()


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
def test_the_model_shows_roles_that_run_ahead(codes):
    """Without rank 1's arrival for what it does not copy, and with stages dealt by task, some order fails."""
    source = protocol.Source()
    if codes:
        source.first_stage = compile("turn", "n0", "eval")
    else:
        source.rank1_arrives, source.counts["k_full"] = False, "1"
    with pytest.raises(protocol.Fault):
        for seed in range(60):
            rng = random.Random(seed)
            protocol.Pair(source, codes, [rng.choice([1, 1, 1, 2, 3, 5]) for _ in range(20)], rng).run()
