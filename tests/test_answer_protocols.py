"""The answering kernels' mbarrier protocols, modelled on the CPU and run under
seeded random interleavings (see tests/protocol_sims): every schedule has to
finish with every read finding what it expects, and each planted mistake has to
be caught by some schedule."""
import random

import pytest

from protocol_sims import prompt_kernel, tree_kernel

CLEAN, PLANTED = 300, 2000
ITEMS = [(0, 0), (1, 1), (2, 2), (3, 3), (5, 5), (1, 2), (0, 1), (2, 3), (1, 0), (4, 5)]
PIECES = [(1, False), (2, False), (3, False), (4, False), (7, False)]
PAIRED = PIECES + [(1, True), (2, True), (3, True), (5, True)]
MODELS = {
    "prompt": (prompt_kernel.run, ITEMS, dict(buffers=2, slots=5), (1, 2, 3, 6)),
    "prompt_64": (prompt_kernel.run, ITEMS, dict(buffers=3, slots=8), (1, 2, 3, 4, 5, 6, 7)),
    "tree": (tree_kernel.run, PIECES, dict(slots=6), (1, 3)),
    "tree_pair": (tree_kernel.run, PAIRED, dict(slots=5), (1, 2, 3)),
}


def draws(n, seed, choices):
    rng = random.Random(seed)
    return [[rng.choice(choices) for _ in range(rng.randint(1, 5))] for _ in range(n)]


@pytest.mark.parametrize("name", sorted(MODELS))
def test_protocol_holds_under_random_schedules(name):
    run, choices, kw, _ = MODELS[name]
    for seed, work in enumerate(draws(CLEAN, 5, choices)):
        run(work, seed, **kw)


@pytest.mark.parametrize("name,mutation", [(n, m) for n in sorted(MODELS) for m in MODELS[n][3]])
def test_planted_protocol_mistake_is_caught(name, mutation):
    run, choices, kw, _ = MODELS[name]
    for seed, work in enumerate(draws(PLANTED, 7, choices)):
        try:
            run(work, seed, mutation=mutation, **kw)
        except AssertionError:
            return
    pytest.fail(f"{name} mutation {mutation} survived {PLANTED} schedules")
