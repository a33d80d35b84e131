"""Token log probabilities against their 64-bit definition.

Tolerances. z = (x - top) / temperature carries two or three fp32 roundings, 2^-22 |z|; each exponential 2^-21 of itself
beside that, sums 2^-20 (fixed trees of a few thousand at most); the logarithm of the sum 2^-20 and its own rounding. A log
probability is z less that: 2^-21 (|z| + 8 + log V). The entropy is a weighted mean of the same numbers: each term's error
times its weight, p |z| at most 1 + log V in all, so 2^-19 (1 + log V) squared covers product and weights.
"""
import numpy as np
import pytest

import kv8_util as ref
from gpu_util import Guarded, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def si():
    import activation_sparse_gb300 as si
    return si


def tdtype(name):
    t = torch()
    return {"bf16": t.bfloat16, "fp16": t.float16, "fp32": t.float32}[name]


def run(si, x, targets=None, K=0, temperature=1.0, entropy=True):
    t = torch()
    N = x.shape[0]
    M = 0 if targets is None else targets.shape[1]
    logp = Guarded((N, M), t.float32) if M else None
    h = Guarded((N,), t.float32) if entropy else None
    top, ids = (Guarded((N, K), t.float32), Guarded((N, K), t.int32)) if K else (None, None)
    si.si_token_logprobs(x, targets=targets, logp=logp.t if M else None, entropy=h.t if entropy else None,
                         top_logp=top.t if K else None, top_ids=ids.t if K else None, temperature=temperature)
    return [None if g is None else g.numpy() for g in (logp, h, top, ids)]


def check(x, targets, K, temperature, got):
    """x float64 [N][V]: what the logits' type holds."""
    logp, h, top, ids = got
    N, V = x.shape
    l, hw = ref.logprobs(x, float(np.float32(temperature)))
    with np.errstate(invalid="ignore"):
        z = np.abs(np.where(np.isfinite(x), x - x.max(-1, keepdims=True), 0) / temperature)
    tol = 2.0 ** -21 * (z + 8 + np.log(V))

    def near(a, b, tol):
        with np.errstate(over="ignore"):  # what no fp32 holds (twice the lowest number) is -inf in it
            b = np.where(np.isinf(b.astype(np.float32)), b.astype(np.float32), b)
        fine = np.isfinite(b)
        assert (np.isnan(a) == np.isnan(b)).all() and (a[~fine & ~np.isnan(b)] == b[~fine & ~np.isnan(b)]).all()
        assert (np.abs(a[fine] - b[fine]) <= tol[fine]).all(), np.abs(a[fine] - b[fine]).max()

    rows = np.arange(N)[:, None]
    if targets is not None:
        on = (targets >= 0) & (targets < V)
        at = np.where(on, targets, 0)
        near(logp, np.where(on, l[rows, at], -np.inf), np.where(on, tol[rows, at], 0))
    if h is not None:
        near(h, hw, np.full(N, 2.0 ** -19 * (1 + np.log(V)) ** 2))
    if K:
        want = ref.best(x, K)
        assert (ids == want).all()
        near(top, l[rows, want], tol[rows, want])


CASES = [
    # N, V, M, K, dtype, temperature, spread
    (1, 1, 1, 1, "fp32", 1.0, 1.0),
    (3, 2, 2, 2, "bf16", 0.5, 1.0),
    (2, 7, 1, 7, "fp16", 2.0, 3.0),
    (5, 31, 3, 20, "fp32", 1.0, 3.0),
    (4, 33, 0, 32, "bf16", 1.0, 0.01),         # nearly all tie
    (300, 257, 1, 5, "bf16", 0.8, 4.0),
    (7, 4096, 4, 8, "fp16", 1.0, 4.0),
    (1, 32768, 1, 32, "fp32", 0.7, 4.0),
    (1, 50001, 2, 4, "bf16", 1.0, 8.0),
    (16, 50001, 2, 32, "fp32", 1.3, 0.1),      # nearly even
    (65, 8191, 1, 1, "fp16", 1.0, 2.0),
    (200, 9999, 1, 3, "bf16", 1.0, 2.0),
    (1, 300007, 8, 32, "bf16", 1.0, 4.0),
    (3, 131072, 1, 0, "fp32", 1.0, 20.0),      # decided
    (700, 5003, 1, 32, "fp32", 1.0, 4.0),
]


@pytest.mark.parametrize("N,V,M,K,dtype,temperature,spread", CASES)
def test_logprobs(si, N, V, M, K, dtype, temperature, spread):
    t = torch()
    rng = np.random.default_rng(V)
    x = t.from_numpy(rng.standard_normal((N, V)) * spread).to(tdtype(dtype)).cuda()
    targets = rng.integers(-1, V + 1, (N, M)).astype(np.int32) if M else None
    got = run(si, x, None if targets is None else t.from_numpy(targets).cuda(), K, temperature)
    check(x.double().cpu().numpy(), targets, K, temperature, got)


@pytest.mark.parametrize("dtype,V", [("bf16", 1003), ("fp16", 4096), ("fp32", 1002), ("bf16", 70001)])
def test_logprobs_of_strided_rows(si, dtype, V):
    """Rows at any element of a wider buffer, its rest full of NaN."""
    t = torch()
    rng = np.random.default_rng(5)
    for off, pad in ((1, 4), (3, 3), (5, 0), (8, 1)):
        wide = t.full((6, V + off + pad), float("nan"), dtype=tdtype(dtype), device="cuda")
        x = wide[:, off:off + V]
        x.copy_(t.from_numpy(rng.standard_normal((6, V)) * 3).cuda())
        targets = rng.integers(0, V, (6, 2)).astype(np.int32)
        check(x.double().cpu().numpy(), targets, 6, 1.0, run(si, x, t.from_numpy(targets).cuda(), 6))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [9, 3001, 90000])
def test_logprobs_of_odd_rows(si, dtype, V):
    """-inf in places, alone, and beside NaN or +inf; the type's lowest and largest; all equal; signed zeros."""
    t = torch()
    rng = np.random.default_rng(7)
    x = rng.standard_normal((12, V)) * 2
    big = float(t.finfo(tdtype(dtype)).max)
    x[0, ::2] = -np.inf
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, V // 2] = 1.5
    x[3, 3] = np.nan
    x[4, V - 1] = np.inf
    x[5] = -np.inf
    x[5, 4] = np.nan
    x[6] = -big
    x[7] = -big
    x[7, 5] = 0.0
    x[8] = 2.25
    x[9] = np.where(np.arange(V) % 2 == 0, -0.0, 0.0)
    x[10] = -big
    x[10, 1] = big
    x[11, 2], x[11, V - 2] = np.inf, np.nan
    g = t.from_numpy(x).to(tdtype(dtype)).cuda()
    targets = np.stack([np.zeros(12), np.full(12, V // 2), np.full(12, 5), np.full(12, -1), np.full(12, V)], 1).astype(np.int32)
    K = min(V, 32)
    check(g.double().cpu().numpy(), targets, K, 1.0, run(si, g, t.from_numpy(targets).cuda(), K))


def test_logprobs_where_the_best_lie_together(si):
    """All of the best in one stretch, and at one thread's places: long runs of candidates."""
    t = torch()
    for V, step in ((40000, 1), (40000, 8), (40000, 2048), (40000, 4096), (150000, 512), (150000, 1024)):
        x = t.zeros(2, V, device="cuda")
        at = (t.arange(32, device="cuda") * step + 3) % V
        x[0, at] = 5.0
        x[1, at] = t.arange(32, device="cuda").float() + 1
        for dtype in (t.float32, t.bfloat16):
            check(x.to(dtype).double().cpu().numpy(), None, 32, 1.0, run(si, x.to(dtype), None, 32))
        y = t.arange(V, device="cuda").float()[None] / V  # rising: the last ones
        check(y.double().cpu().numpy(), None, 32, 1.0, run(si, y, None, 32))
        check((-y).double().cpu().numpy(), None, 32, 1.0, run(si, -y, None, 32))


def test_logprobs_parts_alone_and_no_rows(si):
    t = torch()
    x = t.randn(9, 1234, device="cuda")
    targets = t.randint(0, 1234, (9, 2), device="cuda", dtype=t.int32)
    all_ = run(si, x, targets, 4)
    logp = run(si, x, targets, 0, entropy=False)[0]
    h = run(si, x)[1]
    top = run(si, x, None, 4, entropy=False)
    assert (logp == all_[0]).all() and (h == all_[1]).all() and (top[2] == all_[2]).all() and (top[3] == all_[3]).all()
    si.si_token_logprobs(x[:0], entropy=t.empty(0, device="cuda"))
    si.si_token_logprobs(x)


def test_logprobs_in_a_graph_and_on_another_stream(si):
    t = torch()
    x = t.randn(3, 40001, device="cuda")
    want = run(si, x, None, 8)
    side = t.cuda.Stream()
    h, top, ids = t.zeros(3, device="cuda"), t.zeros(3, 8, device="cuda"), t.zeros(3, 8, dtype=t.int32, device="cuda")
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            for _ in range(3):
                si.si_token_logprobs(x, entropy=h, top_logp=top, top_ids=ids)
        for _ in range(5):
            h.zero_(), ids.zero_()
            g.replay()
    side.synchronize()
    assert (h.cpu().numpy() == want[1]).all() and (top.cpu().numpy() == want[2]).all() and (ids.cpu().numpy() == want[3]).all()


def test_logprobs_past_32_bits(si):
    """Rows whose elements lie past 2^32."""
    t = torch()
    wide = t.empty(3, 2 ** 31 + 64, dtype=t.bfloat16, device="cuda")
    x = wide[:, 33:33 + 5000]
    x.copy_(t.randn(3, 5000, device="cuda"))
    check(x.double().cpu().numpy(), None, 5, 1.0, run(si, x, None, 5))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("temperature", [4.3e-39, 1e-38, 3e38])
def test_logprobs_at_the_ends_of_the_temperature(si, dtype, temperature):
    """The least temperature that is taken: differences become 0, or as large as fp32 holds; and the largest: all even."""
    t = torch()
    rng = np.random.default_rng(8)
    x = t.from_numpy(rng.standard_normal((4, 3001)) * 0.3).to(tdtype(dtype)).cuda()
    x[1, 5], x[1, 2900] = 3.0, 3.0   # two largest
    x[2] = 0.25
    targets = np.tile(np.array([0, 5, 2900], np.int32), (4, 1))
    check(x.double().cpu().numpy(), targets, 8, temperature, run(si, x, t.from_numpy(targets).cuda(), 8, temperature))


def best_of(x, K):
    """Ids of the K largest of every row: NaN first, then by size, then by id."""
    nan = np.isnan(x)
    return np.stack([np.lexsort((np.arange(x.shape[1]), -np.where(n, 0.0, r), ~n))[:K] for r, n in zip(x, nan)])


def check_best(si, g, K):
    """The ids of K alternatives, and their log probabilities by the definition."""
    x = g.double().cpu().numpy()
    top, ids = run(si, g, None, K, entropy=False)[2:]
    want = best_of(x, K)
    assert (ids == want).all()
    check(x, want.astype(np.int32), 0, 1.0, (top, None, None, None))
    return ids


@pytest.mark.parametrize("K", [1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [9, 3001, 90000])
def test_few_alternatives_of_odd_rows(si, K, dtype, V):
    """One alternative has a way of its own: NaN, infinities, ties and signed zeros there, and with two."""
    t = torch()
    rng = np.random.default_rng(9)
    x = rng.standard_normal((13, V)) * 2
    big = float(t.finfo(tdtype(dtype)).max)
    x[0, ::2] = -np.inf
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, V // 2] = 1.5
    x[3, 3] = np.nan
    x[4, V - 1] = np.inf
    x[5] = -np.inf
    x[5, 4] = np.nan
    x[6] = -big
    x[7, V - 2], x[7, V - 1] = np.nan, np.nan
    x[8] = 2.25
    x[9] = np.where(np.arange(V) % 2 == 0, -0.0, 0.0)
    x[10] = -big
    x[10, 1] = big
    x[11, 2], x[11, V - 2] = np.inf, np.nan
    x[12, V // 3], x[12, V - 1] = np.inf, np.inf
    g = t.from_numpy(x).to(tdtype(dtype)).cuda()
    check_best(si, g, K)
    for n in (2, 3, 7, 8):  # a row alone: as many CTAs as a row can have
        check_best(si, g[n:n + 1].contiguous(), K)


@pytest.mark.parametrize("K", [1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_alternatives_that_tie(si, K, dtype):
    """Equal largest logits in other threads, warps, batches and CTAs: the lowest id. Also where they are NaN or -inf."""
    t = torch()
    V = 150001
    for first, step in ((0, 1), (1, 8), (7, 2048), (3, 8192), (18000, 19000), (149990, 1), (5, 512), (16, 16384)):
        at = t.arange(first, min(V, first + 32 * step), step, device="cuda")
        x = t.randn(1, V, device="cuda", generator=t.Generator("cuda").manual_seed(first)).clamp(-4, 4).to(tdtype(dtype))
        for value in (5.0, float("nan"), float("inf")):
            x[0, at] = value
            assert check_best(si, x, K)[0].tolist() == at[:K].tolist()
            for n in (40, 100, 700):  # fewer CTAs a row
                assert (run(si, x.expand(n, V).contiguous(), None, K)[3] == at[:K].cpu().numpy()).all()
    x = t.full((1, V), float("-inf"), dtype=tdtype(dtype), device="cuda")
    assert run(si, x, None, K)[3].tolist() == [list(range(K))]
