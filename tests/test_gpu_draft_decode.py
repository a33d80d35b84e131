"""The example that runs the cache's operators and the sparse FFN together."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

PROMPT = [t * 7 % 24 for t in range(40)]


def test_drafted_trees_give_the_tokens_of_plain_decoding():
    """Without eviction the accepted tokens are the greedy ones, however they were guessed."""
    import draft_decode as ex
    plain, one = ex.decode(ex.Model(), PROMPT, 48, draft=False)
    drafted, more = ex.decode(ex.Model(), PROMPT, 48)
    other, _ = ex.decode(ex.Model(), PROMPT, 48, seed=5)
    assert one == 1.0 and more > 1.0 and len(set(plain)) > 4
    assert drafted == plain and other == plain


def test_the_budget_holds():
    import draft_decode as ex
    model = ex.Model()
    ex.decode(model, PROMPT, 60, budget=50)
    lens = model.cache.lens.cpu()
    assert bool((lens == 50).all())
    table = model.cache.table.sort(-1).values.cpu()
    assert bool((table == table.new_tensor(range(table.shape[-1]))).all())  # still a permutation of the slots
    # the first keys are protected: their slots lead every list
    assert model.cache.table[0, 0, 0, :4].tolist() == [0, 1, 2, 3]
