"""What a call over a cache in 8 bits leaves in its handle."""
import pytest

from gpu_util import torch
from test_gpu_kv import make_rows
from test_gpu_kv8 import Cache8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def si():
    import activation_sparse_gb300 as si
    return si


@pytest.mark.parametrize("streams", [2, 3])
@pytest.mark.parametrize("T,Hq,D", [(1, 4, 128), (4, 8, 64), (2, 4, 256)])
def test_calls_that_ran_at_once_spoil_nothing_later(si, T, Hq, D, streams):
    """Calls of one handle belong on one stream: those that ran on several may have any outputs (the kernel has no wait and
    stays within its scratch whatever the counters hold), and at most the next one meets what they left: the ones after it
    have their own outputs, eager and from a graph."""
    t = torch()
    c = Cache8(si, 71, [3000, 1900, 700], T, 2, D, "bf16")
    q, words, mask = make_rows(c, T, Hq, D, "bf16", "tree" if T > 1 else "none")
    want, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, want, mask=mask, lse=lse)
    side = [t.cuda.Stream() for _ in range(streams)]
    g = t.cuda.CUDAGraph()
    replayed = t.empty_like(q)
    with t.cuda.graph(g):
        si.si_tree_attention(c.kv, q, replayed, mask=mask)
    for _ in range(10):
        t.cuda.synchronize()
        for i in range(20):
            for s in side:
                with t.cuda.stream(s):
                    si.si_tree_attention(c.kv, q, t.empty_like(q), mask=mask)
        t.cuda.synchronize()
        si.si_tree_attention(c.kv, q, t.empty_like(q), mask=mask)  # may still meet what they left
        for _ in range(6):  # more than there are sets of counters
            out, again = t.full_like(q, 7.0), t.empty_like(lse)
            si.si_tree_attention(c.kv, q, out, mask=mask, lse=again)
            assert t.equal(out, want) and t.equal(again, lse)
        replayed.zero_()
        g.replay()
        assert t.equal(replayed, want)


def test_lengths_that_change_between_calls(si):
    """Lists that are cut otherwise from call to call: no call's counters are another's."""
    t = torch()
    c = Cache8(si, 72, [4000, 2500, 90], 2, 2, 128, "bf16")
    q = make_rows(c, 2, 8, 128, "bf16", "none")[0]
    runs = [[4000, 2500, 90], [0, 0, 0], [10, 2500, 1], [4000, 0, 0], [127, 128, 90]]
    wants = []
    for lens in runs:
        c.lens.copy_(t.tensor([lens], dtype=t.int32))
        # a handle of its own each
        kv = si.si_kv_create(c.K, c.V, c.table, c.lens, c.acc, k_scale=c.k_scale, v_scale=c.v_scale, dtype=t.bfloat16)
        wants.append(t.empty_like(q))
        si.si_tree_attention(kv, q, wants[-1])
        kv.close()
    for _ in range(20):
        for lens, want in zip(runs, wants):
            c.lens.copy_(t.tensor([lens], dtype=t.int32))
            out = t.full_like(q, 7.0)
            si.si_tree_attention(c.kv, q, out)
            assert t.equal(out, want)
