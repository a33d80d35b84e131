"""Drafted decoding over a cache of e4m3 codes: what the example does with it, and what it says of its tokens."""
import os
import sys

import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    import draft_decode
    return draft_decode


PROMPT = [t * 7 % 24 for t in range(40)]


def test_drafts_give_plain_tokens(ex):
    a, one = ex.decode(ex.Model(codes=True), PROMPT, 40, draft=False)
    b, more = ex.decode(ex.Model(codes=True), PROMPT, 40, draft=True)
    assert a == b and one == 1.0 and more > 1.0


def test_an_evicting_cache_of_codes_stays_within_its_budget(ex):
    import activation_sparse_gb300 as si
    model = ex.Model(codes=True)
    tokens, _ = ex.decode(model, PROMPT, 100, budget=64)
    assert len(tokens) == 100 and bool((model.cache.lens == 64).all())
    assert si.si_device_error() == 0
    assert bool((model.cache.table.sort(-1).values == torch().arange(512, device="cuda")).all())


@pytest.mark.parametrize("codes", [False, True])
def test_told_log_probabilities(ex, codes):
    """They are those of greedy tokens: at least 1 / vocab each, and not above what the entropy allows."""
    told, told_plain = [], []
    a, _ = ex.decode(ex.Model(codes=codes), PROMPT, 24, told=told)
    b, _ = ex.decode(ex.Model(codes=codes), PROMPT, 24, draft=False, told=told_plain)
    assert a == b and len(told) == len(told_plain) == 24
    for p, h in told + told_plain:
        assert -3.1781 <= p <= 0.0 and -p <= h + 1e-4  # log 24; the likeliest token's -log p is at most the mean of all
