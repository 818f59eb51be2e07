"""The barrier protocols of the decoding passes over a cache, on the CPU:
random interleavings of the models in serving_protocols.py never go wrong, and
leaving out any one wait makes some run fail."""

import random

import pytest

import serving_protocols as models


def own_case(seed):
    rng = random.Random(seed)
    return [rng.choice((1, 1, 2, 3, 5)) for _ in range(rng.randint(1, 5))], rng.choice((3, 4, 5, 6, 8))


def prefix_case(seed):
    rng = random.Random(seed)
    return [(rng.choice((1, 1, 2, 4)), rng.choice((2, 2, 1))) for _ in range(rng.randint(1, 4))], rng.choice((2, 4))


@pytest.mark.parametrize("part", range(4))
def test_own_protocol_holds(part):
    for seed in range(100 * part, 100 * part + 100):
        runs, H = own_case(seed)
        models.run_own(runs, seed, H)


@pytest.mark.parametrize("part", range(4))
def test_prefix_protocol_holds(part):
    for seed in range(100 * part, 100 * part + 100):
        runs, S = prefix_case(seed)
        models.run_prefix(runs, seed, S)


def fails(run, case, seeds, **kw):
    for seed in range(seeds):
        try:
            run(*case(seed)[:1], seed, case(seed)[1], **kw)
        except AssertionError:
            return True
    return False


@pytest.mark.parametrize("name", ["free", "p", "q", "s", "o", "o_end"])
def test_every_wait_of_the_own_protocol_is_needed(name):
    assert fails(models.run_own, own_case, 60, skip=(name,))


@pytest.mark.parametrize("name", ["vfree", "kfree", "q", "p", "s", "fin"])
def test_every_wait_of_the_prefix_protocol_is_needed(name):
    assert fails(models.run_prefix, prefix_case, 60, skip=(name,))


def test_the_last_product_needs_a_barrier_of_its_own():
    """On the scores' barrier the next run's first S can complete a second phase
    before the softmax looks at the first: the wait then never ends."""
    assert fails(models.run_prefix, prefix_case, 200, one_barrier=True)


@pytest.mark.parametrize("part", range(4))
def test_prefix_protocol_holds_where_values_are_hidden(part):
    """The first slot's warps write into V for both slots."""
    for seed in range(100 * part, 100 * part + 100):
        runs, S = prefix_case(seed)
        models.run_prefix(runs, seed, S, scrub=True)


def test_hidden_values_need_their_wait_and_the_first_slot():
    assert fails(models.run_prefix, prefix_case, 60, scrub=True, skip=("scrub",))
    assert fails(models.run_prefix, prefix_case, 60, scrub=True, scrub_slot=1)
