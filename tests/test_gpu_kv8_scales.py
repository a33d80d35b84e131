"""A cache in 8 bits whose scales lie far apart: what a row is given depends on the keys that it weighs alone.

Tolerances. With n keys, p_j the softmax weights and 2^e_j the values' scales: up to 16 rows a key, or above 128
elements, a weight times its value's scale goes into the product as two fp16 terms relative to the largest that its row
has met: the terms lose 2^-22 of it, or 2^-35 of the largest, times a code of up to 448. Else it is rounded once to the
type, relative to the weight (fp16: 2^-35 of the largest weight at least), an fp32 number relative to the row's largest, so
that those below 2^-126 of it are 0. Scores and output as in test_gpu_kv8.py; the
score error is that of the keys which have weight.
"""
import math

import numpy as np
import pytest

import kv8_util as ref8
import kv_util as ref
from gpu_util import torch
from test_gpu_kv import gpu, host, make_rows, score_error, tdtype
from test_gpu_kv8 import Cache8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def si():
    import activation_sparse_gb300 as si
    return si


def weighed(c, q, words, scale):
    """Of every row: the largest weight times its value's scale, the largest value among keys that have weight, and what the
    weights below fp32's normal range give."""
    qh, (K, V, table) = host(q), c.args()
    B, T, Hq, D = qh.shape
    G = Hq // K.shape[1]
    byte = c.v_scale[c.layer].cpu().numpy()
    top, size, least = np.zeros((B, T, Hq, 1)), np.zeros((B, T, Hq, 1)), np.zeros((B, T, Hq, D))
    for b in range(B):
        n = int(c.lens_h[b])
        for h in range(K.shape[1]):
            at = np.arange(n + T) if table is None else table[b, h, :n + T]
            unit = ref8.power(byte[b, h, at // c.block], c.dtype)
            for t in range(T):
                vis = ref.sees(words[b, t], n, T)
                for g in range(h * G, h * G + G if vis.any() else 0):
                    z = scale * (K[b, h, at[vis]] @ qh[b, t, g])
                    p = np.exp(z - z.max())
                    low = p < 2.0 ** -126
                    p /= p.sum()
                    least[b, t, g] = p[low] @ np.abs(V[b, h, at[vis]][low])
                    top[b, t, g] = (p * unit[vis]).max()
                    size[b, t, g] = np.abs(V[b, h, at[vis]])[p > 2.0 ** -100].max()
    return top, size, least


def check(c, q, out, lse, words, scale, light=None):
    """light [B][Hkv][slots]: keys whose weights are 0, so that their scores' errors do not count."""
    K, V, table = c.args()
    want, lse_w, mag = ref.attend(host(q), K, V, table, c.lens_h, words, scale)
    e = score_error(host(q), K if light is None else np.where(light[..., None], 0, K), q.shape[-1], scale) + 2.0 ** -19
    u, n = ref.U[c.dtype], max(c.lens_h) + c.T
    top, size, least = weighed(c, q, words, scale)
    few = q.shape[1] * q.shape[2] // K.shape[1] <= 16 or q.shape[-1] > 128
    if few:
        weights = 2.0 ** -21 * mag + n * 448 * 2.0 ** -35 * top
    else:
        weights = u * mag + least + (n * 2.0 ** -35 * size if c.dtype == "fp16" else 0.0)
    got, lg, empty = host(out), host(lse), words == 0
    assert np.isfinite(got).all()
    bad = np.abs(got - want) - (u * np.abs(want) + weights + 2 * e * mag + (2.0 ** -24 if c.dtype == "fp16" else 1e-37))
    assert bad.max() <= 0, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    assert (np.abs(lg[~empty] - lse_w[~empty]) <= e + 2.0 ** -21 * (1 + np.abs(lse_w[~empty]))).all()
    return want, mag


SHAPES = [(1, 4, 2), (2, 8, 2), (3, 8, 2), (20, 8, 2)]  # T, Hq, Hkv: 2, 8 and 12 rows a key, 80 on the tensor cores' own memory


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("dtype,gap", [("bf16", 30), ("bf16", 40), ("bf16", 120), ("fp16", 22)])
def test_values_of_keys_without_weight(si, T, Hq, Hkv, D, dtype, gap):
    """Keys whose weight is 0 and whose values' scale lies 2^gap above the rest's, early in every warp's share."""
    c = Cache8(si, 61, [700, 90], T, Hkv, D, dtype, spread=0.0)
    q, words, mask = make_rows(c, T, Hq, D, dtype, "tree")
    q[..., 0] = 8.0
    light = np.zeros(c.K.shape[1:4], bool)
    for b in range(2):
        for h in range(Hkv):
            light[b, h, c.table_h[0, b, h, [0, 17, 33, 50, 64, 65]]] = True
    w = gpu(light)[None]
    base = 127 + (-15 if dtype == "fp16" else -7)
    row = torch().zeros(D, dtype=torch().uint8, device="cuda")
    row[0] = 0xFE  # -448
    c.K.view(torch().uint8)[w] = row
    c.k_scale[w] = 127 + 3  # scores of -800 and below
    c.v_scale[c.v_scale != 255] = base
    c.v_scale[w] = base + gap
    out, lse = torch().empty_like(q), torch().empty(q.shape[:3], device="cuda")
    scale = 0.5 / math.sqrt(D)
    si.si_tree_attention(c.kv, q, out, mask=mask, lse=lse, scale=scale)
    check(c, q, out, lse, words, scale, light)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
def test_scales_that_make_up_for_the_weights(si, T, Hq, Hkv, D):
    """Scores that fall as the values' scales rise: every key has about the same part of the output."""
    t = torch()
    c = Cache8(si, 62, [600, 70], T, Hkv, D, "bf16", spread=0.0)
    q, words, mask = make_rows(c, T, Hq, D, "bf16", "tree")
    q *= 0.125
    q[..., 0] = 1.0
    # scores of 1.5 x, x = -24 .. 24 in steps of 4 (exact codes), and scales of 2^-2x: 2^1.5x log2(e) is about as much less
    x = c.rng.integers(-6, 7, c.K.shape[:4]) * 4.0
    c.K.view(t.uint8)[..., 0] = gpu(ref8.encode(x))
    c.k_scale.fill_(127)
    c.K.view(t.uint8)[..., 1:] = gpu(ref8.encode(c.rng.standard_normal(c.K.shape[:4] + (D - 1,)) * 0.25))
    c.v_scale.copy_(gpu((120 - np.round(1.5 * x * math.log2(math.e))).astype(np.uint8)))
    c.V.view(t.uint8).copy_(gpu(ref8.encode(c.rng.standard_normal(c.V.shape) * 100.0)))
    out, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, out, mask=mask, lse=lse, scale=1.5)
    check(c, q, out, lse, words, 1.5)


@pytest.mark.parametrize("n", [0, 29, 300])
@pytest.mark.parametrize("T,Hq,Hkv,D,dtype", [(4, 2, 1, 64, "bf16"), (4, 8, 2, 128, "bf16"), (3, 8, 2, 128, "fp16"), (6, 4, 2, 256, "bf16"),
                                              (20, 8, 2, 128, "bf16")])
def test_values_of_a_node_that_a_row_does_not_see(si, T, Hq, Hkv, D, dtype, n):
    """A sibling's value of an enormous scale: rows that do not see it have what they have beside an ordinary one. The same
    fp32 sums, rescaled at other moments, 2^-19 of the values' weighted size each, and each rounded once."""
    t = torch()
    c = Cache8(si, 63, [n], T, Hkv, D, dtype, spread=0.0)
    words = np.array([[1 << i | 1 for i in range(T)]], np.uint64)  # all children of node 0
    mask = gpu(words.view(np.int64))
    q = gpu(c.rng.standard_normal((1, T, Hq, D)), tdtype(dtype))
    if dtype == "fp16":
        c.v_scale.copy_(t.where(c.v_scale == 255, c.v_scale, c.v_scale - 8))  # 2^-15
    clean, out, lse = t.empty_like(q), t.empty_like(q), t.empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, clean, mask=mask, scale=0.1)
    node = T - 1
    for h in range(Hkv):
        c.v_scale[0, 0, h, int(c.table_h[0, 0, h, n + node])] += 22 if dtype == "fp16" else 100
    si.si_tree_attention(c.kv, q, out, mask=mask, lse=lse, scale=0.1)
    want, mag = check(c, q, out, lse, words, 0.1)
    few = T * Hq // Hkv <= 16 or D > 128
    near = 2.0 ** -18 * mag + 2 * ref.U[dtype] * np.abs(want) + (2.0 ** -24 if dtype == "fp16" else 0.0) if few else 0.0
    assert (np.abs(host(out) - host(clean)) <= near)[0, :node].all()


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 2, 64), (2, 8, 2, 128), (3, 8, 2, 128), (3, 4, 2, 256), (20, 8, 2, 64), (40, 4, 1, 128)])
def test_queries_near_the_types_largest(si, T, Hq, Hkv, D):
    """Queries 2^121 times as large over keys 2^-121 as large have the same scores, outputs and weights, to the bit: nothing
    between the product and the score leaves fp32's range."""
    t = torch()
    c = Cache8(si, 64, [400], T, Hkv, D, "bf16", spread=0.0)
    q, words, mask = make_rows(c, T, Hq, D, "bf16", "tree")
    q[0, 0, 0, 1:] = 0.0  # an element alone
    got = []
    for up in (0, 121):
        c.k_scale[c.k_scale != 255] = 124 - up  # 2^-3 and 2^-124
        big = q * 2.0 ** up
        assert bool(big.isfinite().all())
        out, lse, acc = t.empty_like(q), t.empty(q.shape[:3], device="cuda"), t.zeros_like(c.acc[0])
        si.si_tree_attention(c.kv, big, out, mask=mask, lse=lse, scale=0.02)
        si.si_kv_accumulate(c.kv, big, lse, mask=mask, scale=0.02, acc_out=acc)
        got.append((out, lse, acc))
    assert bool(got[0][1].isfinite().all())
    for x, y in zip(*got):
        assert t.equal(x, y)


@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 2, 64), (2, 8, 2, 128), (4, 8, 2, 128), (2, 4, 2, 256), (20, 8, 2, 128)])
def test_scores_that_rise_as_scales_fall_along_the_list(si, T, Hq, Hkv, D, falling):
    """Every few tiles a score outgrows the ones before it by little while the scales fall as much, or the other way round:
    what has been summed is rescaled over and over, and no key's part is lost."""
    t = torch()
    c = Cache8(si, 65, [5200, 900], T, Hkv, D, "bf16", spread=0.0)
    q, words, mask = make_rows(c, T, Hq, D, "bf16", "none" if T == 1 else "tree")
    q *= 0.125
    q[..., 0] = 1.0
    # scores of 0.5 x, x the codes from -448 to 448 in order, and scales of about 2^-(0.5 x log2(e) / 5): 2^+-65
    codes = np.sort(ref8.CODES[~np.isnan(ref8.CODES)])
    c.K.view(t.uint8)[..., 1:] = gpu(ref8.encode(c.rng.standard_normal(c.K.shape[:4] + (D - 1,)) * 0.25))
    c.V.view(t.uint8).copy_(gpu(ref8.encode(c.rng.standard_normal(c.V.shape) * 100.0)))
    c.k_scale.fill_(127)
    x = np.zeros(c.K.shape[:4])
    for b, n in enumerate(c.lens_h + T):
        rise = codes[np.linspace(0, len(codes) - 1, n).astype(int)] / 5  # -89.6 .. 89.6
        for h in range(Hkv):
            x[0, b, h, c.table_h[0, b, h, :n]] = rise[::-1] if falling else rise
    x = ref8.CODES[ref8.encode(x)]
    c.K.view(t.uint8)[..., 0] = gpu(ref8.encode(x))
    c.v_scale.copy_(gpu((120 - np.round(0.5 * x * math.log2(math.e))).astype(np.uint8)))
    out, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, out, mask=mask, lse=lse, scale=0.5)
    check(c, q, out, lse, words, 0.5)
