"""The key/value cache's operators against their 64-bit definitions.

Tolerances. U is half a rounding step of the cache's type, relative (bf16
2^-8, fp16 2^-11).
 - append: one rounding of a value whose fp32 terms (two products of inputs
   with cos and sin, each good to 2^-22) carry 2^-21 (|a| + |b|).
 - attention: each weight is rounded once (U) before the product with v, the
   output once more (U), so U (sum p |v| + |o|); the fp32 score error e moves
   every weight by a factor exp(+-e), numerator and denominator, 2 e in all.
   A score is scale times D products summed in fp32, D / 16 + 8 roundings of
   2^-23 (truncation in the tensor cores) relative to the products' absolute
   sum; exp2 and the running rescale add 2^-19.
   fp16 weights below 2^-14 of the row's largest lose up to 2^-25 each: the
   sum of |v| times 2^-25 covers it.
 - lse: e and 2^-21 of its own size.  weights: exp(e) and the lse given.
"""
import math

import numpy as np
import pytest

import kv_util as ref
from gpu_util import Guarded, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def si():
    import activation_sparse_gb300 as si
    return si


def tdtype(name):
    return {"bf16": torch().bfloat16, "fp16": torch().float16}[name]


def gpu(a, dtype=None):
    t = torch().from_numpy(np.array(a, order="C")).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A cache of random keys and values with free slots full of NaN."""

    def __init__(self, si, seed, lens, T, Hkv, D, dtype, table=True, slack=0, L=1, layer=0, k_scale=1.0):
        t = torch()
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.T, self.layer, self.lens_h = T, layer, np.array(lens)
        cap = max(lens) + T + slack
        slots = cap + (7 if table else 0)
        self.table_h = ref.tables(rng, (L, B, Hkv), cap, slots) if table else None
        K, V = (t.full((L, B, Hkv, slots, D), float("nan"), dtype=tdtype(dtype), device="cuda") for _ in range(2))
        for b in range(B):
            for h in range(Hkv):
                n = lens[b] + T
                at = gpu(np.arange(n) if not table else self.table_h[layer, b, h, :n].astype(np.int64))
                K[layer, b, h, at] = gpu(k_scale * rng.standard_normal((n, D)), tdtype(dtype))
                V[layer, b, h, at] = gpu(rng.standard_normal((n, D)), tdtype(dtype))
        self.K, self.V = K, V
        self.table = gpu(self.table_h) if table else None
        self.lens = gpu(np.broadcast_to(np.array(lens, np.int32), (L, B)))
        self.acc = gpu(rng.random((L, B, Hkv, slots)), t.float32)
        self.kv = si.si_kv_create(K, V, self.table, self.lens, self.acc)
        self.rng = rng

    def args(self):
        return (host(self.K[self.layer]), host(self.V[self.layer]),
                None if self.table_h is None else self.table_h[self.layer])


def score_error(q, K, D, scale):
    """Bound of a score's fp32 error: (D / 16 + 8) 2^-23 of the largest absolute product sum."""
    k = np.nan_to_num(np.abs(K))
    big = max(np.abs(q).reshape(-1, D).sum(-1).max() * k.max(), 1e-30)
    exact = np.sqrt((q ** 2).sum(-1).max()) * np.sqrt((k ** 2).sum(-1).max())  # Cauchy-Schwarz on absolute values
    return scale * (D / 16 + 8) * 2.0 ** -23 * min(big, exact)


def check_attend(c, q, out, lse, words, scale, dtype):
    K, V, table = c.args()
    qh = host(q)
    D = qh.shape[-1]
    Kz = K
    want, lse_w, mag = ref.attend(qh, Kz, V, table, c.lens_h, words, scale)
    e = score_error(qh, K, D, scale) + 2.0 ** -19
    u = ref.U[dtype]
    vmax = np.nan_to_num(np.abs(V)).max()
    tiny = 2.0 ** -25 * (max(c.lens_h) + c.T) * vmax if dtype == "fp16" else 0.0
    got = host(out)
    assert np.isfinite(got).all()
    tol = u * (mag + np.abs(want)) + 2 * e * mag + tiny + 2.0 ** -24
    bad = np.abs(got - want) - tol
    assert bad.max() <= 0, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    empty = words == 0
    assert (got[empty] == 0).all()
    if lse is not None:
        lg = host(lse)
        assert np.isneginf(lg[empty]).all()
        assert (np.abs(lg[~empty] - lse_w[~empty]) <= e + 2.0 ** -21 * (1 + np.abs(lse_w[~empty]))).all()


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("B,T,Hq,Hkv,D,pairs,axes,inter,dtype,table", [
    (1, 1, 32, 8, 64, 32, 1, False, "bf16", True),
    (2, 5, 6, 3, 128, 64, 3, False, "fp16", True),
    (3, 17, 4, 2, 80, 40, 2, True, "bf16", True),
    (1, 3, 2, 1, 256, 128, 4, False, "bf16", False),
    (2, 2, 5, 5, 96, 16, 1, True, "fp16", True),     # a partial rotation, interleaved
    (1, 70, 8, 2, 128, 32, 1, False, "bf16", True),  # a partial rotation, split
    (1, 2, 0, 2, 16, 8, 1, False, "fp16", False),    # no queries
])
def test_append(si, B, T, Hq, Hkv, D, pairs, axes, inter, dtype, table):
    t = torch()
    L, layer = 2, 1
    c = Cache(si, 11, [3] * B, T, Hkv, D, dtype, table=table, slack=4, L=L, layer=layer)
    rng = c.rng
    inv = 10000.0 ** (-np.arange(pairs) / pairs)
    axis = rng.integers(0, axes, pairs)
    axis[0], axis[-1] = axes - 1, 0
    rope = si.si_rope_create(D, inv_freq=inv, axis=axis, interleaved=inter)
    pos = rng.integers(0, 5000, (B, T, rope.n_axes))
    pos[0, 0], pos[-1, -1] = 2147483647, -2147483648
    qkv = gpu(rng.standard_normal((B, T, Hq + 2 * Hkv + 1, D)), tdtype(dtype))  # slices of a wider projection
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:Hq + 2 * Hkv]
    K0, V0, acc0 = c.K.clone(), c.V.clone(), c.acc.clone()
    q_out = Guarded((B, T, max(Hq, 1), D), tdtype(dtype))
    si.si_kv_append(c.kv, rope, q if Hq else None, k, v, gpu(pos.astype(np.int32)), q_out.t if Hq else None, layer=layer)
    cos, sin = ref.angles(pos, inv, axis)
    u = ref.U[dtype]

    def near(got, x):
        want = ref.rotate(x, cos, sin, inter)
        size = np.abs(x[..., :2 * pairs]).max(-1, keepdims=True) * 2
        assert (np.abs(got - want) <= u * np.abs(want) + 2.0 ** -21 * size + 2.0 ** -25).all()
        assert (got[..., 2 * pairs:] == x[..., 2 * pairs:]).all()

    if Hq:
        q_out.check()
        near(host(q_out.t), host(q))
    written = np.zeros(c.K.shape[:4], bool)
    kk, vv = np.empty((B, T, Hkv, D)), np.empty((B, T, Hkv, D))
    for b in range(B):
        for h in range(Hkv):
            at = np.arange(3, 3 + T) if not table else c.table_h[layer, b, h, 3:3 + T]
            written[layer, b, h, at] = True
            kk[b, :, h], vv[b, :, h] = host(c.K[layer, b, h])[at], host(c.V[layer, b, h])[at]
    near(kk, host(k))
    assert (vv == host(v)).all()
    w = gpu(written)
    for new, old in ((c.K, K0), (c.V, V0)):
        assert t.equal(new.view(t.int16)[~w], old.view(t.int16)[~w])
    assert t.equal(c.acc[~w], acc0[~w]) and bool((c.acc[w] == 0).all())


def test_append_in_place_queries(si):
    c = Cache(si, 12, [0], 4, 2, 64, "bf16")
    rope = si.si_rope_create(64)
    q = gpu(c.rng.standard_normal((1, 4, 4, 64)), tdtype("bf16"))
    k = gpu(c.rng.standard_normal((1, 4, 2, 64)), tdtype("bf16"))
    pos = gpu(np.arange(4, dtype=np.int32).reshape(1, 4, 1))
    apart = torch().empty_like(q)
    si.si_kv_append(c.kv, rope, q, k, k, pos, apart)
    si.si_kv_append(c.kv, rope, q, k, k, pos, q)
    assert torch().equal(q, apart)


def test_append_out_of_bounds_is_refused(si):
    """A full sequence writes nothing; the other one is served; a bad table entry writes nothing."""
    t = torch()
    c = Cache(si, 13, [2, 2], 2, 2, 64, "bf16")
    c.lens.copy_(gpu(np.array([[2, 3]], np.int32)))  # sequence 1 has one free entry for two tokens
    c.table[0, 0, 1, 2] = 1 << 28
    K0 = c.K.clone()
    rope = si.si_rope_create(64)
    k = gpu(c.rng.standard_normal((2, 2, 2, 64)), tdtype("bf16"))
    si.si_kv_append(c.kv, rope, None, k, k, t.zeros(2, 2, 1, dtype=t.int32, device="cuda"), None)
    assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE
    same = (c.K.view(t.int16) == K0.view(t.int16)).all(-1)
    assert bool(same[0, 1].all())
    assert (~same[0, 0, 0]).sum() == 2 and (~same[0, 0, 1]).sum() == 1


# ---------------------------------------------------------------- attention

CASES = [
    # lens, T, Hq, Hkv, D, dtype, table, mask
    ([0], 1, 1, 1, 64, "bf16", True, "none"),
    ([1], 1, 4, 2, 128, "fp16", False, "none"),
    ([62], 1, 8, 2, 64, "bf16", True, "tree"),
    ([63], 1, 8, 2, 64, "bf16", True, "none"),
    ([64], 1, 3, 3, 64, "fp16", True, "none"),
    ([1000], 1, 16, 2, 128, "bf16", True, "none"),
    ([5000], 1, 8, 1, 128, "fp16", False, "none"),
    ([130, 0, 700], 5, 6, 2, 128, "bf16", True, "tree"),
    ([60, 61, 127], 7, 9, 3, 96, "fp16", True, "tree"),
    ([33, 500], 16, 8, 4, 80, "bf16", True, "pad"),
    ([100, 3], 64, 4, 1, 128, "fp16", True, "pad"),
    ([2000], 33, 14, 2, 128, "bf16", True, "tree"),
    ([90, 700], 64, 8, 1, 64, "bf16", False, "none"),
    ([300], 3, 10, 2, 256, "bf16", True, "tree"),
    ([65, 64], 20, 8, 2, 256, "fp16", True, "pad"),
    ([40], 2, 2, 1, 8, "bf16", True, "tree"),
    ([17] * 30, 2, 4, 2, 64, "fp16", True, "tree"),
    ([3000, 1], 64, 16, 2, 128, "bf16", True, "pad"),
    ([0, 63, 64, 128], 9, 8, 2, 128, "bf16", True, "tree"),
    ([4000], 40, 5, 1, 64, "fp16", True, "pad"),
    ([1500], 17, 3, 3, 128, "fp16", False, "tree"),
    ([5, 70] * 100, 1, 4, 2, 64, "bf16", True, "none"),       # more lists than CTAs
    ([3, 130] * 100, 5, 8, 2, 64, "fp16", True, "pad"),
    ([9000, 1, 64, 7000, 20], 40, 8, 2, 128, "bf16", False, "tree"),
]


def make_rows(c, T, Hq, D, dtype, mask):
    rng, B = c.rng, len(c.lens_h)
    q = gpu(rng.standard_normal((B, T, Hq, D)), tdtype(dtype))
    if mask == "none":
        return q, ref.chain(B, T), None
    nodes = [max(0, T - 3 * b - (1 if T > 1 else 0)) for b in range(B)] if mask == "pad" else None
    words = ref.trees(rng, B, T, nodes)
    return q, words, gpu(words.view(np.int64))


@pytest.mark.parametrize("lens,T,Hq,Hkv,D,dtype,table,mask", CASES)
def test_attention(si, lens, T, Hq, Hkv, D, dtype, table, mask):
    c = Cache(si, 21, lens, T, Hkv, D, dtype, table=table, L=2, layer=1)
    q, words, mask_t = make_rows(c, T, Hq, D, dtype, mask)
    # what padding nodes hold never matters
    for b in range(len(lens)):
        for node in range(T):
            if not any(int(w) >> node & 1 for w in words[b]):
                for h in range(Hkv):
                    slot = lens[b] + node if not table else int(c.table_h[1, b, h, lens[b] + node])
                    c.K[1, b, h, slot] = float("nan")
                    c.V[1, b, h, slot] = float("inf")
                q[b, node] = float("nan")
    out, lse = Guarded(q.shape, q.dtype), Guarded(q.shape[:3], torch().float32)
    scale = 1.3 / math.sqrt(D)
    si.si_tree_attention(c.kv, q, out.t, mask=mask_t, lse=lse.t, scale=scale, layer=1)
    out.check(), lse.check()
    qz = torch().nan_to_num(q.float()).to(q.dtype)
    check_attend(c, qz, out.t, lse.t, words, scale, dtype)
    again = torch().empty_like(q)
    si.si_tree_attention(c.kv, q, again, mask=mask_t, scale=scale, layer=1)
    assert torch().equal(again, out.t)  # no lse asked for, and the same bits


@pytest.mark.parametrize("T,Hq,Hkv", [(64, 32, 8), (16, 16, 4), (1, 8, 2)])
def test_attention_back_to_back(si, T, Hq, Hkv):
    """Launches that overlap their neighbours' ends, by the hundred: the same bits and no wait that runs out."""
    t = torch()
    c = Cache(si, 29, [3000, 1900, 700], T, Hkv, 128, "bf16")
    q, words, mask = make_rows(c, T, Hq, 128, "bf16", "tree" if T > 1 else "none")
    want, outs = t.empty_like(q), [t.empty_like(q) for _ in range(4)]
    si.si_tree_attention(c.kv, q, want, mask=mask)
    for _ in range(100):
        for o in outs:
            si.si_tree_attention(c.kv, q, o, mask=mask)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        for _ in range(25):
            for o in outs:
                si.si_tree_attention(c.kv, q, o, mask=mask)
    for _ in range(4):
        g.replay()
    t.cuda.synchronize()
    assert all(t.equal(o, want) for o in outs)


def rise_late(c, q, Hkv, D, at_nodes, last=400, slope=0.1):
    """Scores of the chosen nodes' rows climb by `slope` a key over each list's last `last` keys: maxima that
    outgrow the ones of the tiles before, in some warps and not in others."""
    u = np.zeros(D)
    u[::2] = (2.0 / D) ** 0.5
    for b, n in enumerate(c.lens_h):
        climb = slope * D ** 0.5 / 8.0 * np.maximum(0, np.arange(n) - n + last)
        for h in range(Hkv):
            slots = gpu(np.arange(n) if c.table_h is None else c.table_h[0, b, h, :n].astype(np.int64))
            k = host(c.K[0, b, h, slots])
            k -= np.outer(k @ u, u)
            c.K[0, b, h, slots] = gpu(k + np.outer(climb, u), c.K.dtype)
    x = host(q)
    x -= (x @ u)[..., None] * u
    x[:, at_nodes] += 8.0 * u
    q.copy_(gpu(x, q.dtype))


@pytest.mark.parametrize("lens,T,Hq,Hkv,D,dtype,table", [
    ([3000, 1900, 700], 64, 32, 8, 128, "bf16", True),
    ([3001, 1920, 640, 65], 16, 16, 2, 128, "fp16", True),
    ([1500, 130, 900], 33, 8, 2, 64, "bf16", False),
    ([100] * 40, 24, 8, 2, 64, "fp16", True),        # a CTA has lists of two tiles
])
def test_attention_every_launch_with_maxima_that_rise_late(si, lens, T, Hq, Hkv, D, dtype, table):
    """Rows that rescale in a list's last tiles beside rows that do not; every one of many overlapping launches is
    looked at, not the last into a buffer."""
    t = torch()
    c = Cache(si, 61, lens, T, Hkv, D, dtype, table=table)
    q, words, mask = make_rows(c, T, Hq, D, dtype, "tree")
    per_warp = max(1, 32 // (Hq // Hkv))
    rise_late(c, q, Hkv, D, [n for n in range(T) if n // per_warp % 2])
    want, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, want, mask=mask, lse=lse)
    check_attend(c, q, want, lse, words, D ** -0.5, dtype)
    outs = [t.zeros_like(q) for _ in range(120)]
    for o in outs:
        si.si_tree_attention(c.kv, q, o, mask=mask)
    assert all(t.equal(o, want) for o in outs)
    for o in outs:
        o.zero_()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        for o in outs:
            si.si_tree_attention(c.kv, q, o, mask=mask)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        assert all(t.equal(o, want) for o in outs)


def test_attention_between_prefill_products(si):
    """Tree attention and the FFN's prefill product, which both take tensor memory, in turn without a pause: every
    launch gives its bits and no wait runs out."""
    t = torch()
    c = Cache(si, 62, [700, 300], 64, 2, 128, "bf16")
    q, words, mask = make_rows(c, 64, 8, 128, "bf16", "tree")
    rng = np.random.default_rng(63)
    W = [gpu(rng.standard_normal(s) / 16, t.bfloat16) for s in ((1024, 256), (1024, 256), (256, 1024))]
    score = gpu(rng.random(1024), t.float32)
    layer = si.si_pack_loaded(*W, score, score, 0.7, 0.4)
    X = gpu(rng.standard_normal((300, 256)), t.bfloat16)
    n = si.si_count(0.5, 1024)
    pairs = [(t.zeros_like(q), t.zeros(1, n, dtype=t.int32, device="cuda"), t.zeros(300, layer.n_pad, device="cuda")) for _ in range(60)]

    def both():
        for o, S, A in pairs:
            si.si_select_dynamic(layer, X, 300, 1, 200, 0.5, S, A)
            si.si_tree_attention(c.kv, q, o, mask=mask)

    both()
    want, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, want, mask=mask, lse=lse)
    check_attend(c, q, want, lse, words, 128 ** -0.5, "bf16")
    S0, A0 = pairs[0][1].clone(), pairs[0][2].clone()
    assert all(t.equal(o, want) and t.equal(S, S0) and t.equal(A, A0) for o, S, A in pairs)
    for x in pairs:
        for y in x:
            y.zero_()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        both()
    g.replay()
    assert all(t.equal(o, want) and t.equal(S, S0) and t.equal(A, A0) for o, S, A in pairs)
    layer.close()


def test_attention_peaked_and_flat_rows(si):
    """Scores far apart (one key takes all) and all equal."""
    c = Cache(si, 22, [700], 1, 1, 64, "bf16", k_scale=8.0)
    q = gpu(4.0 * c.rng.standard_normal((1, 1, 4, 64)), tdtype("bf16"))
    q[0, 0, 3] = 0
    out, lse = torch().empty_like(q), torch().empty(1, 1, 4, device="cuda")
    si.si_tree_attention(c.kv, q, out, lse=lse)
    check_attend(c, q, out, lse, ref.chain(1, 1), 64 ** -0.5, "bf16")


@pytest.mark.parametrize("heads", [1, 32])  # few rows a key, and many
def test_attention_lowest_values_and_infinities(si, heads):
    """Keys of the type's lowest value weigh nothing beside others and share evenly among
    themselves; a key at minus infinity is not there; a row of those alone is empty."""
    t = torch()
    K = t.zeros(1, 3, 1, 4, 64, dtype=t.bfloat16, device="cuda")
    V = t.ones(1, 3, 1, 4, 64, dtype=t.bfloat16, device="cuda")
    low = t.finfo(t.bfloat16).min
    K[0, 0, 0, 0, 0], K[0, 1, 0, :, 0], K[0, 2, 0, :, 0] = low, low, -math.inf
    V[0, 0, 0, 0] = 5.0
    V[0, 1, 0, 0] = 5.0
    kv = si.si_kv_create(K, V, None, t.full((1, 3), 3, dtype=t.int32, device="cuda"))
    q = t.zeros(3, 1, heads, 64, dtype=t.bfloat16, device="cuda")
    q[:, :, :, 0] = 1
    out, lse = t.empty_like(q), t.empty(3, 1, heads, device="cuda")
    si.si_tree_attention(kv, q, out, lse=lse, scale=0.5)
    assert bool((out[0] == 1).all()) and bool((out[1] == 2).all()) and bool((out[2] == 0).all())
    assert bool(((lse[0] - math.log(3)).abs() < 1e-6).all()) and bool((lse[2] == -math.inf).all())


@pytest.mark.parametrize("dtype,D,T,Hq", [("bf16", 128, 6, 1), ("fp16", 64, 40, 4), ("bf16", 256, 6, 2), ("fp16", 128, 64, 8)])
def test_attention_odd_values_stay_with_their_branch(si, dtype, D, T, Hq):
    """Infinities and NaN in a drafted node's key and value reach the rows that see it and no other."""
    t = torch()
    c = Cache(si, 23, [50], T, 1, D, dtype)
    words = ref.trees(c.rng, 1, T)
    sick = {1: (3, math.inf), 4: (D - 1, math.nan), T - 1: (0, -math.inf)}
    clean = c.V.clone()
    for node, (d, value) in sick.items():
        c.V[0, 0, 0, int(c.table_h[0, 0, 0, 50 + node]), d] = value
    c.K[0, 0, 0, int(c.table_h[0, 0, 0, 50 + 2]), 5] = math.nan
    q = gpu(c.rng.standard_normal((1, T, Hq, D)), tdtype(dtype))
    out = t.empty_like(q)
    si.si_tree_attention(c.kv, q, out, mask=gpu(words.view(np.int64)))
    ok = np.ones((T, D), bool)
    for i in range(T):
        for node, (d, _) in sick.items():
            if int(words[0, i]) >> node & 1:
                ok[i, d] = False
        if int(words[0, i]) >> 2 & 1:
            ok[i] = False
    got = host(out)[0].transpose(0, 2, 1)  # [T, D, Hq]
    assert np.isfinite(got[ok]).all() and not np.isfinite(got[~ok]).any()
    # the healthy elements are what they are without the others
    c.V.copy_(clean)
    c.K[0, 0, 0, int(c.table_h[0, 0, 0, 50 + 2]), 5] = 0
    base = t.empty_like(q)
    si.si_tree_attention(c.kv, q, base, mask=gpu(words.view(np.int64)))
    assert (host(base)[0].transpose(0, 2, 1)[ok] == got[ok]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,T,G,Hkv,D", [
    (3000, 1, 4, 1, 64), (3000, 2, 8, 1, 128), (3000, 3, 4, 1, 256), (3000, 8, 4, 1, 128), (3000, 40, 4, 1, 64),
    (400, 1, 2, 320, 64), (400, 2, 2, 160, 256), (400, 6, 3, 320, 64)])  # whole lists in a block
@pytest.mark.parametrize("place,above", [(0.0, 9.0), (0.0, 12.3), (0.0, 14.2), (0.5, 14.2), (1.0, 12.3)])
def test_attention_one_key_takes_nearly_all(si, dtype, n, T, G, Hkv, D, place, above):
    """One key far above the others and with a value of 0: the output is what the others give, each with a weight
    far below the largest, as exact as the type."""
    t = torch()
    at = int(place * (n - 1))
    rng = np.random.default_rng(64)
    K, V = (t.zeros(1, 1, Hkv, n + T, D, dtype=tdtype(dtype), device="cuda") for _ in range(2))
    V[0, 0, :, :n] = gpu(1 + rng.random((Hkv, n, D)) / 4, V.dtype)
    K[0, 0, :, at, 0], V[0, 0, :, at] = above, 0
    kv = si.si_kv_create(K, V, None, t.full((1, 1), n, dtype=t.int32, device="cuda"))
    q = t.zeros(1, T, Hkv * G, D, dtype=tdtype(dtype), device="cuda")
    q[..., 0] = gpu(1 - 0.0625 * (np.arange(Hkv * G) % G), q.dtype)
    out, lse = t.empty_like(q), t.empty(1, T, Hkv * G, device="cuda")
    si.si_tree_attention(kv, q, out, lse=lse, scale=1.0)
    want, lse_w, mag = ref.attend(host(q), host(K[0]), host(V[0]), None, [n], ref.chain(1, T), 1.0)
    e = (D / 16 + 8) * 2.0 ** -23 * above + 2.0 ** -19
    tol = ref.U[dtype] * (mag + np.abs(want)) + 2 * e * mag + 2.0 ** -30
    if dtype == "fp16":
        tol += 2.0 ** -25 * (np.abs(want) < 2.0 ** -13)  # an output below the type's normal range
    assert (np.abs(host(out) - want) <= tol).all(), (np.abs(host(out) - want) / mag).max()
    assert (np.abs(host(lse) - lse_w) <= e + 2.0 ** -21 * (1 + np.abs(lse_w))).all()


@pytest.mark.parametrize("lens,T,Hq,Hkv,D,dtype,table", [
    ([40], 1, 8, 2, 64, "bf16", True),
    ([1000], 1, 32, 8, 64, "bf16", True),
    ([130, 7, 700], 4, 8, 2, 128, "bf16", True),
    ([20], 16, 2, 2, 128, "bf16", False),
    ([64], 2, 16, 2, 80, "fp16", True),
    ([100, 30], 4, 8, 2, 256, "bf16", True),
    ([5000], 1, 8, 1, 128, "fp16", False),
])
def test_attention_few_rows_rounds_the_output_alone(si, lens, T, Hq, Hkv, D, dtype, table):
    """Up to 16 rows a key: a weight is carried in two terms of the type, so it is good to
    U^2 and what is left is the output's own rounding. Sums in fp32: an addition a step of sixteen keys."""
    t = torch()
    c = Cache(si, 65, lens, T, Hkv, D, dtype, table=table)
    q, words, mask = make_rows(c, T, Hq, D, dtype, "tree")
    out = t.empty_like(q)
    si.si_tree_attention(c.kv, q, out, mask=mask)
    K, V, tab = c.args()
    want, _, mag = ref.attend(host(q), K, V, tab, c.lens_h, words, D ** -0.5)
    u, n = ref.U[dtype], max(lens) + T
    e = score_error(host(q), K, D, D ** -0.5) + 2.0 ** -19
    err = (u * u + 2 * e + (n / 16 + 16) * 2.0 ** -23) * mag
    tol = u * (np.abs(want) + err) + err + 2.0 ** -25
    assert (np.abs(host(out) - want) <= tol).all(), (np.abs(host(out) - want) - tol).max()


def test_attention_strides(si):
    """Keys and values inside one interleaved pool, queries inside a fused projection."""
    t = torch()
    rng = np.random.default_rng(24)
    B, Hkv, D, n, T = 2, 2, 64, 90, 3
    pool = gpu(rng.standard_normal((B, n + T, 2, Hkv, D + 8)), t.float16)  # [seq][slot][k or v][head][D + pad]
    K, V = (pool[:, :, i, :, :D].permute(0, 2, 1, 3)[None] for i in (0, 1))
    wide = gpu(rng.standard_normal((B, T, 9, D)), t.float16)
    q = wide[:, :, 3:7]
    kv = si.si_kv_create(K, V, None, gpu(np.array([[n, n - 40]], np.int32)))
    out = t.empty(B, T, 4, D, dtype=t.float16, device="cuda")
    si.si_tree_attention(kv, q, out)
    plain = si.si_kv_create(K.contiguous(), V.contiguous(), None, gpu(np.array([[n, n - 40]], np.int32)))
    want = t.empty_like(out)
    si.si_tree_attention(plain, q.contiguous(), want)
    assert t.equal(out, want)


def test_strides_of_single_elements(si):
    """One sequence and one token whose strides there mean nothing, as tensors from elsewhere have them: the same bits."""
    t = torch()
    D, n = 64, 30
    rng = np.random.default_rng(66)
    rope = si.si_rope_create(D)

    def step(odd):
        """The result with plain strides, or with 1 and 3 in the places that do not matter."""
        like = lambda x: x.as_strided(x.shape, [(1, 3)[i % 2] if k == 1 else s for i, (k, s) in enumerate(zip(x.shape, x.stride()))]) if odd else x  # noqa: E731
        K, V = (like(gpu(kv0[i], t.bfloat16)) for i in (0, 1))
        acc = like(t.zeros(1, 1, 2, n + 1, device="cuda"))
        table = like(gpu(np.arange(n + 1, dtype=np.int32)[::-1] + np.zeros((1, 1, 2, 1), np.int32)).to(t.int32))
        lens = gpu(np.array([[n]], np.int32))
        kv = si.si_kv_create(K, V, table, lens, acc)
        q, k, v = (like(gpu(x, t.bfloat16)) for x in new)
        qr, out, lse = t.empty(1, 1, 4, D, dtype=t.bfloat16, device="cuda"), t.empty(1, 1, 4, D, dtype=t.bfloat16, device="cuda"), t.empty(1, 1, 4, device="cuda")
        si.si_kv_append(kv, rope, q, k, v, t.full((1, 1, 1), 7, dtype=t.int32, device="cuda"), qr)
        si.si_tree_attention(kv, like(qr), out, lse=lse)
        more = like(t.zeros(1, 2, n + 1, device="cuda"))
        si.si_kv_accumulate(kv, like(qr), lse, acc_out=more)
        si.si_kv_accumulate(kv, like(qr), lse)
        si.si_kv_evict(kv, 1, 20, sinks=1, recent=2)
        return [x.contiguous() for x in (K, V, qr, out, lse, more, acc, table, lens)]

    kv0 = rng.standard_normal((2, 1, 1, 2, n + 1, D))
    new = [rng.standard_normal((1, 1, h, D)) for h in (4, 2, 2)]
    for a, b in zip(step(False), step(True)):
        assert t.equal(a, b)


@pytest.mark.parametrize("D,pad", [(64, 0), (64, 8), (128, 0), (128, 64), (96, 0)])
def test_attention_strides_many_rows(si, D, pad):
    """The same with trees of many rows: heads side by side in a slot, with and without room between them."""
    t = torch()
    rng = np.random.default_rng(28)
    B, Hkv, n, T, Hq = 2, 3, 200, 12, 12
    pool = gpu(rng.standard_normal((B, n + T, 2, Hkv, D + pad)), t.bfloat16)
    K, V = (pool[:, :, i, :, :D].permute(0, 2, 1, 3)[None] for i in (0, 1))
    q = gpu(rng.standard_normal((B, T, Hq + 5, D)), t.bfloat16)[:, :, 2:2 + Hq]
    lens = [n, n - 77]
    table = ref.tables(rng, (1, B, Hkv), n + T, n + T)
    kv = si.si_kv_create(K, V, gpu(table), gpu(np.array([lens], np.int32)))
    out, lse = t.empty(B, T, Hq, D, dtype=t.bfloat16, device="cuda"), t.empty(B, T, Hq, device="cuda")
    words = ref.trees(rng, B, T)
    si.si_tree_attention(kv, q, out, mask=gpu(words.view(np.int64)), lse=lse)
    want, lse_w, mag = ref.attend(host(q), host(K[0]), host(V[0]), table[0], lens, words, D ** -0.5)
    assert (np.abs(host(out) - want) <= 2.0 ** -8 * (mag + np.abs(want)) * 1.01 + 1e-5).all()
    assert np.abs(host(lse) - lse_w).max() < 1e-5


def test_attention_shared_pool(si):
    """One pool for all sequences: sequence stride 0, lists without common slots."""
    t = torch()
    rng = np.random.default_rng(25)
    B, Hkv, D, n = 3, 2, 128, 70
    pool_k, pool_v = (gpu(rng.standard_normal((1, 1, Hkv, B * (n + 1), D)), t.bfloat16) for _ in range(2))
    table = np.stack([rng.permutation(B * (n + 1)).reshape(B, n + 1) for _ in range(Hkv)], 1)[None].astype(np.int32)
    lens = np.full((1, B), n, np.int32)
    kv = si.si_kv_create(pool_k.expand(1, B, -1, -1, -1), pool_v.expand(1, B, -1, -1, -1), gpu(table), gpu(lens))
    q = gpu(rng.standard_normal((B, 1, 4, D)), t.bfloat16)
    out = t.empty_like(q)
    si.si_tree_attention(kv, q, out)
    Kh, Vh = (np.broadcast_to(host(p[0]), (B, Hkv, B * (n + 1), D)) for p in (pool_k, pool_v))
    want, _, mag = ref.attend(host(q), Kh, Vh, table[0], lens[0], ref.chain(B, 1), D ** -0.5)
    assert (np.abs(host(out) - want) <= 2.0 ** -8 * (mag + np.abs(want)) * 1.01 + 1e-5).all()


def test_attention_far_slots(si):
    """Element offsets past 2^31: the first and the last slots of a 2^25-slot pool."""
    t = torch()
    n_slots, D = (1 << 25) + 3, 64
    K, V = (t.empty(1, 1, 1, n_slots, D, dtype=t.bfloat16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(26)
    slots = np.array([0, n_slots - 1, 5, n_slots - 7, 1 << 24, n_slots - 2], np.int32)
    idx = gpu(slots.astype(np.int64))
    kh, vh = gpu(rng.standard_normal((6, D)), t.bfloat16), gpu(rng.standard_normal((6, D)), t.bfloat16)
    K[0, 0, 0, idx], V[0, 0, 0, idx] = kh, vh
    acc = t.zeros(1, 1, 1, n_slots, device="cuda")
    kv = si.si_kv_create(K, V, gpu(slots.reshape(1, 1, 1, 6)), t.full((1, 1), 5, dtype=t.int32, device="cuda"), acc)
    q = gpu(rng.standard_normal((1, 1, 1, D)), t.bfloat16)
    out, lse = t.empty_like(q), t.empty(1, 1, 1, device="cuda")
    si.si_tree_attention(kv, q, out, lse=lse)
    args = host(q), host(kh)[None, None], host(vh)[None, None]
    want, lse_w, mag = ref.attend(*args, None, [5], ref.chain(1, 1), D ** -0.5)
    assert (np.abs(host(out) - want) <= 2.0 ** -8 * (mag + np.abs(want)) * 1.01 + 1e-5).all()
    si.si_kv_accumulate(kv, q, lse)
    p = ref.weigh(args[0], args[1], None, [5], ref.chain(1, 1), None, host(lse), np.zeros((1, 1, 6)), D ** -0.5)
    assert np.abs(host(acc[0, 0, 0, idx]) - p[0, 0]).max() < 1e-5
    rope = si.si_rope_create(D)
    k = gpu(rng.standard_normal((1, 1, 1, D)), t.bfloat16)
    si.si_kv_append(kv, rope, None, k, k, t.zeros(1, 1, 1, dtype=t.int32, device="cuda"), None)
    assert t.equal(K[0, 0, 0, n_slots - 2], k[0, 0, 0])


def test_attention_out_of_bounds_gives_zeros(si):
    c = Cache(si, 27, [20, 20], 2, 1, 64, "bf16")
    q = gpu(c.rng.standard_normal((2, 2, 2, 64)), tdtype("bf16"))
    good = torch().empty_like(q)
    si.si_tree_attention(c.kv, q, good)
    c.lens.copy_(gpu(np.array([[20, 21]], np.int32)))
    out, lse = torch().ones_like(q), torch().empty(2, 2, 2, device="cuda")
    si.si_tree_attention(c.kv, q, out, lse=lse)
    assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE
    assert torch().equal(out[0], good[0]) and not out[1].any() and bool(torch().isneginf(lse[1]).all())
    c.lens.fill_(-1)
    si.si_tree_attention(c.kv, q, out)
    assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE and not out.any()
    c.lens.fill_(20)
    c.table[0, 0, 0, 3] = -5
    si.si_tree_attention(c.kv, q, out)
    assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("lens,T,Hq,Hkv,D,dtype,table,mask", CASES)
@pytest.mark.parametrize("rows", ["all", "some"])
def test_accumulate(si, lens, T, Hq, Hkv, D, dtype, table, mask, rows):
    t = torch()
    c = Cache(si, 31, lens, T, Hkv, D, dtype, table=table, L=2, layer=1)
    q, words, mask_t = make_rows(c, T, Hq, D, dtype, mask)
    K, V, tab = c.args()
    scale = 1.3 / math.sqrt(D)
    _, lse, _ = ref.attend(host(q), np.nan_to_num(K), np.nan_to_num(V), tab, c.lens_h, words, scale)
    lse32 = lse.astype(np.float32)
    picked = None if rows == "all" else np.array([sum(1 << i for i in range(b % 2, T, 3)) for b in range(len(lens))], np.uint64)
    acc0 = c.acc.clone()
    out = Guarded((len(lens), Hkv, c.K.shape[3]), t.float32, fill=-1)
    rows_t = None if picked is None else gpu(picked.view(np.int64))
    si.si_kv_accumulate(c.kv, q, gpu(lse32), mask=mask_t, rows=rows_t, scale=scale, acc_out=out.t, layer=1)
    out.check()
    assert t.equal(c.acc, acc0)
    want = ref.weigh(host(q), np.nan_to_num(K), tab, c.lens_h, words, picked, lse32.astype(np.float64), host(acc0[1]), scale)
    listed = np.zeros(want.shape, bool)
    for b in range(len(lens)):
        for h in range(Hkv):
            n = lens[b] + T
            listed[b, h, np.arange(n) if tab is None else tab[b, h, :n]] = True
    got = host(out.t)
    assert (got[~listed] == -1).all()
    e = score_error(host(q), K, D, scale) + 2.0 ** -20 * (1 + np.abs(lse[np.isfinite(lse)]).max())
    size = want - host(acc0[1])
    tol = size * e * 1.1 + (T * Hq // Hkv + 2) * 2.0 ** -24 * want + 1e-30
    assert (np.abs(got - want)[listed] <= tol[listed]).all(), (np.abs(got - want) - tol)[listed].max()
    # in place, with the same bits
    si.si_kv_accumulate(c.kv, q, gpu(lse32), mask=mask_t, rows=rows_t, scale=scale, layer=1)
    w = gpu(listed)
    assert t.equal(c.acc[1][w], out.t[w]) and t.equal(c.acc[1][~w], acc0[1][~w]) and t.equal(c.acc[0], acc0[0])


def test_accumulate_infinite_keys(si):
    """A key with an infinity weighs nothing where its score is minus infinity; rows that are not there do not change that."""
    t = torch()
    K = t.zeros(1, 1, 1, 70, 64, dtype=t.bfloat16, device="cuda")
    K[0, 0, 0, 3, 0] = -math.inf
    acc = t.zeros(1, 1, 1, 70, device="cuda")
    kv = si.si_kv_create(K, K, None, t.full((1, 1), 69, dtype=t.int32, device="cuda"), acc)
    q = t.ones(1, 1, 3, 64, dtype=t.bfloat16, device="cuda")
    out, lse = t.empty_like(q), t.empty(1, 1, 3, device="cuda")
    si.si_tree_attention(kv, q, out, lse=lse)
    si.si_kv_accumulate(kv, q, lse)
    want = t.full((70,), 3 / 69, device="cuda")
    want[3] = 0
    assert t.allclose(acc[0, 0, 0], want, rtol=1e-5, atol=0)


@pytest.mark.parametrize("heads", [1, 32])  # lse from the kernel for few rows a key, and for many
@pytest.mark.parametrize("scale", [0.5, 0.3, 64 ** -0.5 * 1.1])
def test_accumulate_lowest_values(si, heads, scale):
    """Weights of keys of the type's lowest value: nothing beside others, finite and alike among themselves (a
    32-bit lse of that size cannot hold how many they are), nothing in a row of minus infinities."""
    t = torch()
    K = t.zeros(1, 3, 1, 4, 64, dtype=t.bfloat16, device="cuda")
    low = t.finfo(t.bfloat16).min
    K[0, 0, 0, 0, 0], K[0, 1, 0, :, 0], K[0, 2, 0, :, 0] = low, low, -math.inf
    acc = t.zeros(1, 3, 1, 4, device="cuda")
    kv = si.si_kv_create(K, t.ones_like(K), None, t.full((1, 3), 3, dtype=t.int32, device="cuda"), acc)
    q = t.zeros(3, 1, heads, 64, dtype=t.bfloat16, device="cuda")
    q[:, :, :, 0] = 1
    out, lse = t.empty_like(q), t.empty(3, 1, heads, device="cuda")
    si.si_tree_attention(kv, q, out, lse=lse, scale=scale)
    si.si_kv_accumulate(kv, q, lse, scale=scale)
    got = acc[0, :, 0].cpu()
    assert bool(t.isfinite(got).all())
    assert got[0, 0] == 0 and bool(((got[0, 1:] - heads / 3).abs() < 1e-5 * heads).all())
    assert bool((got[1] == got[1, 0]).all()) and heads / 4 <= float(got[1, 0]) <= heads
    assert bool((got[2] == 0).all())


def test_attention_weights_sum_to_rows(si):
    """The weights of one call's own lse add up to the number of its rows."""
    c = Cache(si, 32, [777], 9, 2, 128, "bf16")
    q, words, mask = make_rows(c, 9, 8, 128, "bf16", "tree")
    out, lse = torch().empty_like(q), torch().empty(1, 9, 8, device="cuda")
    si.si_tree_attention(c.kv, q, out, mask=mask, lse=lse)
    c.acc.zero_()
    si.si_kv_accumulate(c.kv, q, lse, mask=mask)
    assert np.allclose(host(c.acc).sum(-1), 9 * 4, rtol=1e-5)


# ----------------------------------------------------------------- eviction

def run_evict(si, table, lens, acc, T, path, n_path, budget, sinks, recent, in_place, layer=None):
    t = torch()
    L, B, H, cap = table.shape
    K = t.zeros(L, B, H, acc.shape[3], 8, dtype=t.bfloat16, device="cuda")
    tab, ln = Guarded(table.shape, t.int32), Guarded(lens.shape, t.int32)
    tab.t.copy_(gpu(table)), ln.t.copy_(gpu(lens.astype(np.int32)))
    kv = si.si_kv_create(K, K, tab.t, ln.t, gpu(acc, t.float32))
    args = dict(sinks=sinks, recent=recent, path=None if path is None else gpu(path.astype(np.int32)),
                n_path=None if n_path is None else gpu(n_path.astype(np.int32)), layer=layer)
    if in_place:
        si.si_kv_evict(kv, T, budget, **args)
        return tab.numpy(), ln.numpy()
    to, lo = Guarded(table.shape, t.int32, fill=-9), Guarded(lens.shape, t.int32, fill=-9)
    si.si_kv_evict(kv, T, budget, table_out=to.t, len_out=lo.t, **args)
    assert (tab.numpy() == table).all() and (ln.numpy() == lens).all()
    return to.numpy(), lo.numpy()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("L,B,H,lens,T,path,budget,sinks,recent,weights", [
    (1, 1, 1, [0], 1, False, 4, 0, 0, "real"),
    (1, 1, 2, [9], 0, False, 4, 1, 1, "real"),
    (1, 2, 2, [9, 3], 1, False, 4, 1, 1, "real"),
    (2, 2, 3, [50, 40], 8, True, 32, 4, 8, "real"),
    (3, 2, 2, [700, 33], 16, True, 256, 0, 64, "ties"),
    (1, 1, 4, [3000], 64, True, 2999, 4, 100, "real"),
    (1, 2, 1, [5000, 5000], 1, False, 1024, 4, 1020, "real"),   # nothing but sinks and recent
    (1, 1, 2, [4096], 5, True, 1, 0, 0, "real"),
    (1, 1, 2, [4097], 200, False, 1500, 2, 9, "zero"),
    (1, 1, 1, [40000], 3, True, 30000, 4, 512, "close"),
    (1, 1, 1, [190000], 1, False, 100001, 4, 512, "real"),
    (1, 2, 2, [300, 200], 7, True, 0, 0, 0, "real"),            # acceptance alone
    (1, 2, 2, [300, 200], 7, False, 1000, 0, 0, "real"),        # a budget that is not met
    (1, 2, 2, [300, 200], 7, True, 0, 2147483647, 2147483647, "real"),  # sinks and recent mean nothing without one
    (2, 1, 2, [900], 7, False, 700, 350, 350, "real"),          # budget taken by sinks and recent
    (2, 1, 2, [9000], 7, False, 7000, 3000, 3000, "ties"),
    (1, 1, 2, [2500], 1, False, 1200, 0, 3, "odd"),
    (40, 3, 2, [64, 65, 66], 4, True, 64, 1, 4, "ties"),
])
def test_evict(si, in_place, L, B, H, lens, T, path, budget, sinks, recent, weights):
    rng = np.random.default_rng(41)
    cap = max(lens) + T + 3
    slots = cap + 5
    table = ref.tables(rng, (L, B, H), cap, slots)
    lens = np.broadcast_to(np.array(lens, np.int32), (L, B)).copy()
    lens -= (np.arange(L)[:, None] % 2 * (lens > 5)).astype(np.int32)  # layers may differ
    acc = np.exp(2 * rng.standard_normal((L, B, H, slots))).astype(np.float32)
    if weights == "ties":
        acc = rng.integers(0, 3, acc.shape).astype(np.float32)
    elif weights == "zero":
        acc[:] = 0
        acc[..., ::2] = -0.0
    elif weights == "close":  # keys that differ in the last bits alone
        acc = (np.float32(1).view(np.int32) + rng.integers(0, 700, acc.shape).astype(np.int32)).view(np.float32)
    elif weights == "odd":
        acc[rng.random(acc.shape) < .2] = np.nan
        acc[rng.random(acc.shape) < .1] = np.inf
        acc[rng.random(acc.shape) < .1] *= -1
        acc[rng.random(acc.shape) < .1] = -np.inf
        neg = np.isnan(acc) & (rng.random(acc.shape) < .5)
        acc[neg] = np.uint32(0xFFC00001).view(np.float32)
    p = n_path = None
    if path:
        p = np.stack([rng.permutation(T) for _ in range(B)])
        n_path = rng.integers(0, T + 1, B)
    elif T > 1:
        n_path = np.array([T - 1 - b for b in range(B)])
    want_t, want_n = ref.evict(table, lens, acc, T, p, n_path, budget, sinks, recent)
    got_t, got_n = run_evict(si, table, lens, acc, T, p, n_path, budget, sinks, recent, in_place)
    assert (got_n == want_n).all()
    assert (got_t == want_t).all(), np.argwhere(got_t != want_t)[:5]
    assert (np.sort(got_t, -1) == np.sort(table, -1)).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("L,B,H,lens,T,budget,sinks,recent,weights", [
    (40, 4, 3, [40, 7, 0, 64], 5, 32, 2, 4, "real"),
    (40, 4, 3, [300, 1030, 290, 900], 1, 256, 4, 16, "ties"),
    (60, 2, 4, [1500, 2100], 16, 1400, 0, 100, "odd"),
    (60, 1, 8, [4900], 3, 4500, 4, 512, "real"),
    (20, 2, 2, [6500, 3000], 3, 2500, 4, 512, "ties"),
])
def test_evict_many_lists(si, in_place, L, B, H, lens, T, budget, sinks, recent, weights):
    """More lists than CTAs of one kind run at once, and lists that few CTAs share."""
    rng = np.random.default_rng(44)
    cap = max(lens) + T + 3
    table = ref.tables(rng, (L, B, H), cap, cap)
    lens = np.broadcast_to(np.array(lens, np.int32), (L, B)).copy()
    acc = np.exp(2 * rng.standard_normal((L, B, H, cap))).astype(np.float32)
    if weights == "ties":
        acc = np.floor(acc)
    elif weights == "odd":
        acc[rng.random(acc.shape) < .1] = np.nan
        acc[rng.random(acc.shape) < .1] = -np.inf
    path = np.stack([rng.permutation(T) for _ in range(B)])
    n_path = rng.integers(0, T + 1, B)
    want_t, want_n = ref.evict(table, lens, acc, T, path, n_path, budget, sinks, recent)
    got_t, got_n = run_evict(si, table, lens, acc, T, path, n_path, budget, sinks, recent, in_place)
    assert (got_n == want_n).all()
    assert (got_t == want_t).all(), np.argwhere(got_t != want_t)[:5]


def test_evict_one_layer(si):
    rng = np.random.default_rng(42)
    table = ref.tables(rng, (3, 2, 2), 60, 60)
    lens = np.full((3, 2), 50, np.int32)
    acc = rng.random((3, 2, 2, 60)).astype(np.float32)
    want_t, want_n = ref.evict(table, lens, acc, 2, None, None, 30, 1, 3)
    for in_place in (True, False):
        got_t, got_n = run_evict(si, table, lens, acc, 2, None, None, 30, 1, 3, in_place, layer=1)
        assert (got_t[1] == want_t[1]).all() and (got_n[1] == want_n[1]).all()
        rest_t, rest_n = (table, lens) if in_place else (np.full_like(table, -9), np.full_like(lens, -9))
        assert (got_t[[0, 2]] == rest_t[[0, 2]]).all() and (got_n[[0, 2]] == rest_n[[0, 2]]).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_bad_paths_and_lengths(si, in_place):
    rng = np.random.default_rng(43)
    B, T = 6, 4
    table = ref.tables(rng, (1, B, 2), 40, 40)
    lens = np.array([[30, 30, 30, 30, 37, -1]], np.int32)  # the last two are out of bounds
    acc = rng.random((1, B, 2, 40)).astype(np.float32)
    path = np.array([[0, 2, 3, 1], [1, 1, 0, 0], [0, 4, 0, 0], [0, 1, 2, 3], [0, 1, 2, 3], [0, 1, 2, 3]])
    n_path = np.array([3, 2, 2, 5, 2, 2])
    ok = np.array([3, 0, 0, 0, 0, 0])  # a path that is not valid accepts nothing
    safe = lens.copy()
    safe[0, 4:] = 30
    want_t, want_n = ref.evict(table, safe, acc, T, path, ok, 20, 2, 4)
    got_t, got_n = run_evict(si, table, lens, acc, T, path, n_path, 20, 2, 4, in_place)
    assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE | si.SI_DEVERR_COUNT
    assert (got_t[:, :4] == want_t[:, :4]).all() and (got_n[:, :4] == want_n[:, :4]).all()
    assert (got_t[:, 4:] == table[:, 4:]).all() and (got_n[:, 4:] == lens[:, 4:]).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bad", [[-1, -2, -3, -4], [-9, -2147483648, -40, -1], [38, 41, 2147483647, 39]])
def test_evict_lengths_out_of_bounds_touch_nothing(si, in_place, bad):
    """Lists out of bounds, between good ones and with paths that are valid and permuted: no entry of any other
    list changes, and the bad lists and lengths are what they were."""
    rng = np.random.default_rng(45)
    B, T, cap = 9, 4, 40
    table = ref.tables(rng, (1, B, 2), cap, cap)
    lens = np.full((1, B), 30, np.int32)
    lens[0, 1::2] = bad
    acc = rng.random((1, B, 2, cap)).astype(np.float32)
    path = np.array([[2, 0, 3, 1]] * B)
    n_path = np.full(B, 3)
    safe = np.where(np.arange(B) % 2, 0, 30).astype(np.int32)[None]
    want_t, want_n = ref.evict(table, safe, acc, T, path, n_path, 20, 2, 4)
    want_t[0, 1::2], want_n[0, 1::2] = table[0, 1::2], lens[0, 1::2]
    for budget, expect in ((20, (want_t, want_n)), (0, None)):
        if expect is None:  # acceptance alone
            expect = ref.evict(table, safe, acc, T, path, n_path, 0, 0, 0)
            expect[0][0, 1::2], expect[1][0, 1::2] = table[0, 1::2], lens[0, 1::2]
        got_t, got_n = run_evict(si, table, lens, acc, T, path, n_path, budget, 2, 4, in_place)
        assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE
        assert (got_t == expect[0]).all(), np.argwhere(got_t != expect[0])[:5]
        assert (got_n == expect[1]).all()


# ------------------------------------------------------------ streams, graphs

def test_step_on_another_stream_and_in_a_graph(si):
    """append -> attention -> weights -> eviction, eager, on a side stream and replayed from a graph: the same bits."""
    t = torch()

    def build():
        c = Cache(si, 51, [40, 25], 4, 2, 64, "bf16", slack=8)
        rng = np.random.default_rng(52)
        q = gpu(rng.standard_normal((2, 4, 4, 64)), t.bfloat16)
        k, v = (gpu(rng.standard_normal((2, 4, 2, 64)), t.bfloat16) for _ in range(2))
        words = gpu(ref.trees(rng, 2, 4).view(np.int64))
        pos = gpu(np.arange(4, dtype=np.int32).reshape(1, 4, 1).repeat(2, 0) + 40)
        n_path = gpu(np.array([2, 1], np.int32))
        path = gpu(np.array([[0, 2, 0, 0], [3, 0, 0, 0]], np.int32))
        rows = gpu(np.array([5, 8], np.int64))
        rope = si.si_rope_create(64)
        qr, out, lse = t.empty_like(q), t.empty_like(q), t.empty(2, 4, 4, device="cuda")

        def step():
            si.si_kv_append(c.kv, rope, q, k, v, pos, qr)
            si.si_tree_attention(c.kv, qr, out, mask=words, lse=lse)
            si.si_kv_accumulate(c.kv, qr, lse, mask=words, rows=rows)
            si.si_kv_evict(c.kv, 4, 30, sinks=2, recent=4, path=path, n_path=n_path)

        return c, step, (out, lse, c.table, c.lens, c.acc)

    c0, step0, res0 = build()
    for _ in range(3):
        step0()
    want = [x.clone() for x in res0]
    c1, step1, res1 = build()
    side = t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(side):
        for _ in range(3):
            step1()
    side.synchronize()
    c2, step2, res2 = build()
    state = [x.clone() for x in (c2.K, c2.V, c2.table, c2.lens, c2.acc)]
    t.cuda.synchronize()
    with t.cuda.stream(side):
        step2()  # the scratch is made before the capture
    side.synchronize()
    for x, y in zip((c2.K, c2.V, c2.table, c2.lens, c2.acc), state):
        x.copy_(y)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step2()
    for _ in range(3):
        g.replay()
    t.cuda.synchronize()
    for a, b, d in zip(want, res1, res2):
        assert t.equal(a.view(t.uint8), b.view(t.uint8)) and t.equal(a.view(t.uint8), d.view(t.uint8))
    assert int(c0.lens[0, 0]) == 30


def test_scratch_does_not_grow_in_a_capture(si):
    t = torch()
    c = Cache(si, 53, [10], 1, 1, 64, "bf16")
    q = t.zeros(1, 1, 1, 64, dtype=t.bfloat16, device="cuda")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        with pytest.raises(si.SIError, match="before capture"):
            si.si_tree_attention(c.kv, q, t.empty_like(q))
        with pytest.raises(si.SIError, match="before capture"):
            si.si_kv_evict(c.kv, 1, 4)


@pytest.mark.parametrize("D,small,large", [(128, (1, 8), (16, 32)), (64, (2, 4), (64, 64)), (256, (1, 2), (40, 8))])
def test_graphs_outlive_larger_calls(si, D, small, large):
    """A graph of a small call gives its bits after larger calls on its handle; the larger one needs no more
    scratch, so that it can be captured at once."""
    t = torch()
    c = Cache(si, 54, [4000], 64, 2, D, "bf16")

    def call(T, Hq, seed):
        q = gpu(np.random.default_rng(seed).standard_normal((1, T, Hq, D)), t.bfloat16)
        out, lse = t.zeros_like(q), t.zeros(1, T, Hq, device="cuda")
        return (lambda: si.si_tree_attention(c.kv, q, out, lse=lse)), out, lse

    one, out1, lse1 = call(*small, 55)
    many, out2, lse2 = call(*large, 56)
    one()
    want1 = out1.clone(), lse1.clone()
    graphs = t.cuda.CUDAGraph(), t.cuda.CUDAGraph()
    with t.cuda.graph(graphs[0]):
        one()
    with t.cuda.graph(graphs[1]):
        many()
    many()
    want2 = out2.clone(), lse2.clone()
    for o in (out1, lse1, out2, lse2):
        o.zero_()
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    assert t.equal(out1, want1[0]) and t.equal(lse1, want1[1])
    assert t.equal(out2, want2[0]) and t.equal(lse2, want2[1])
