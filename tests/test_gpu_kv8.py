"""The operators over a cache in 8 bits against their 64-bit definitions.

Tolerances. What a slot holds is exact (a code times a power of two, a number of the cache's type), so attention and
weights are compared with the definition over those numbers, with the bounds of the cache in 16 bits (see
test_gpu_kv.py): weights rounded once to the type, one rounding of the output, the scores' fp32 error. Weights that
go into the product as two fp16 terms, with the largest scale that a warp has met as their unit, lose less than 2^-35
of the largest value each: n times that.
Codes: a code is within half a step of its value over the scale: 2^-4 of it, and 2^-10 where it is below the normal
range; the value carries the rotation's fp32 error, 2^-21 (|a| + |b|). Scales: the least power of two for a largest
magnitude that is 2^-20 larger or smaller.
"""
import math

import numpy as np
import pytest

import kv8_util as ref8
import kv_util as ref
from gpu_util import Guarded, torch
from test_gpu_kv import check_attend, gpu, host, make_rows, score_error, tdtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def si():
    import activation_sparse_gb300 as si
    return si


def bytes_of(t):
    return t.view(torch().uint8).cpu().numpy()


class Cache8:
    """A cache of random codes, rows of many sizes; free slots hold NaN codes and NaN scales."""

    def __init__(self, si, seed, lens, T, Hkv, D, dtype, block=1, table=True, slack=0, L=1, layer=0, spread=2.0, n_slots=None, acc=True):
        t = torch()
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.T, self.layer, self.lens_h, self.dtype, self.block = T, layer, np.array(lens), dtype, block
        cap = max(lens) + T + slack
        slots = n_slots or cap + (7 if table else 0)
        self.table_h = ref.tables(rng, (L, B, Hkv), cap, slots) if table else None
        nb = -(-slots // block)
        code = [np.full((L, B, Hkv, slots, D), 0x7F, np.uint8) for _ in range(2)]
        byte = [np.full((L, B, Hkv, nb), 255 if block == 1 else 127, np.uint8) for _ in range(2)]
        for b in range(B):
            for h in range(Hkv):
                n = lens[b] + T
                at = np.arange(n) if not table else self.table_h[layer, b, h, :n]
                for c, e in zip(code, byte):
                    x = rng.standard_normal((n, D))
                    c[layer, b, h, at] = ref8.encode(x * 100.0)
                    # about 1 in size: 100 of a scale of 2^-7, times a spread
                    size = np.clip(np.round(120 + spread * rng.standard_normal(nb)), *(127 + np.array(ref8.LIMITS[dtype])))
                    e[layer, b, h, at // block] = size[at // block]
        self.set(si, code, byte, lens, gpu(rng.random((L, B, Hkv, slots)), t.float32) if acc else None, L)
        self.rng = rng

    def set(self, si, code, byte, lens, acc, L):
        t = torch()
        self.K, self.V = (gpu(c).view(t.float8_e4m3fn) for c in code)
        self.k_scale, self.v_scale = (gpu(e) for e in byte)
        self.table = gpu(self.table_h) if self.table_h is not None else None
        self.lens = gpu(np.broadcast_to(np.array(lens, np.int32), (L, len(lens))))
        self.acc = acc
        self.kv = si.si_kv_create(self.K, self.V, self.table, self.lens, self.acc, k_scale=self.k_scale, v_scale=self.v_scale,
                                  block=self.block, dtype=tdtype(self.dtype))

    def values(self, which):
        return ref8.decode(bytes_of(getattr(self, which)[self.layer]), bytes_of(getattr(self, which.lower() + "_scale")[self.layer]),
                           self.dtype, self.block)

    def args(self):
        return self.values("K"), self.values("V"), None if self.table_h is None else self.table_h[self.layer]

    def hide(self, words):
        """What nodes that nobody sees hold never matters."""
        for b in range(len(self.lens_h)):
            for node in range(self.T):
                if any(int(w) >> node & 1 for w in words[b]):
                    continue
                for h in range(self.K.shape[2]):
                    slot = self.lens_h[b] + node if self.table is None else int(self.table_h[self.layer, b, h, self.lens_h[b] + node])
                    for pool in (self.K, self.V):
                        pool.view(torch().uint8)[self.layer, b, h, slot] = 0x7F


def check(c, q, out, lse, words, scale, dtype):
    """check_attend's bounds over what the codes stand for; bf16 gets the room of fp16 terms too."""
    want_tiny = 2.0 ** -35 * (max(c.lens_h) + c.T) * np.nan_to_num(np.abs(c.values("V"))).max()
    K, V, table = c.args()
    want, lse_w, mag = ref.attend(host(q), K, V, table, c.lens_h, words, scale)
    e = score_error(host(q), K, q.shape[-1], scale) + 2.0 ** -19
    u, got = ref.U[dtype], host(out)
    assert np.isfinite(got).all()
    least = 2.0 ** -24 if dtype == "fp16" else 0.0  # the type's least number
    tiny = 2.0 ** -25 * (max(c.lens_h) + c.T) * np.nan_to_num(np.abs(V)).max() if dtype == "fp16" else want_tiny
    bad = np.abs(got - want) - (u * (mag + np.abs(want)) + 2 * e * mag + tiny + least + 1e-37)
    assert bad.max() <= 0, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    empty = words == 0
    assert (got[empty] == 0).all()
    if lse is not None:
        lg = host(lse)
        assert np.isneginf(lg[empty]).all()
        assert (np.abs(lg[~empty] - lse_w[~empty]) <= e + 2.0 ** -21 * (1 + np.abs(lse_w[~empty]))).all()


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("B,T,Hq,Hkv,D,pairs,axes,inter,dtype,table,block", [
    (1, 1, 32, 8, 64, 32, 1, False, "bf16", True, 1),
    (2, 5, 6, 3, 128, 64, 3, False, "fp16", True, 1),
    (3, 17, 4, 2, 80, 40, 2, True, "bf16", True, 1),
    (1, 3, 2, 1, 256, 128, 4, False, "bf16", False, 1),
    (2, 2, 5, 5, 96, 16, 1, True, "fp16", True, 1),     # a partial rotation, interleaved
    (1, 70, 8, 2, 256, 8, 1, False, "bf16", True, 1),   # the least rotation of the widest head
    (1, 2, 0, 2, 16, 8, 1, False, "fp16", False, 1),    # no queries
    (2, 33, 8, 8, 128, 64, 1, True, "fp16", True, 1 << 20),
    (1, 9, 4, 40, 64, 32, 1, False, "bf16", True, 4),   # more rows than the block has groups
    (1, 6, 2, 33, 112, 56, 1, False, "bf16", False, 16),
])
def test_append(si, B, T, Hq, Hkv, D, pairs, axes, inter, dtype, table, block):
    t = torch()
    L, layer = 2, 1
    c = Cache8(si, 11, [3] * B, T, Hkv, D, dtype, block=block, table=table, slack=4, L=L, layer=layer)
    rng = c.rng
    inv = 10000.0 ** (-np.arange(pairs) / pairs)
    axis = rng.integers(0, axes, pairs)
    axis[0], axis[-1] = axes - 1, 0
    rope = si.si_rope_create(D, inv_freq=inv, axis=axis, interleaved=inter)
    pos = rng.integers(0, 5000, (B, T, rope.n_axes))
    pos[0, 0], pos[-1, -1] = 2147483647, -2147483648
    # slices of a wider projection, rows from tiny to large; one of zeros
    x = rng.standard_normal((B, T, Hq + 2 * Hkv + 1, D)) * 2.0 ** rng.integers(-9, 9, (B, T, Hq + 2 * Hkv + 1, 1))
    x[0, 0, Hq] = 0.0
    x[0, 0, -2] = 0.0
    qkv = gpu(x, tdtype(dtype))
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:Hq + 2 * Hkv]
    before = [bytes_of(a).copy() for a in (c.K, c.V, c.k_scale, c.v_scale)]
    acc0 = c.acc.clone()
    q_out = Guarded((B, T, max(Hq, 1), D), tdtype(dtype))
    si.si_kv_append(c.kv, rope, q if Hq else None, k, v, gpu(pos.astype(np.int32)), q_out.t if Hq else None, layer=layer)
    cos, sin = ref.angles(pos, inv, axis)
    if Hq:
        q_out.check()
        qh = host(q)
        want = ref.rotate(qh, cos, sin, inter)
        size = np.abs(qh[..., :2 * pairs]).max(-1, keepdims=True) * 2
        assert (np.abs(host(q_out.t) - want) <= ref.U[dtype] * np.abs(want) + 2.0 ** -21 * size + 2.0 ** -25).all()
    written = np.zeros(c.K.shape[:4], bool)
    touched = np.zeros(c.k_scale.shape, bool)
    lo, hi = ref8.LIMITS[dtype]
    for pool, scale, rows in (("K", "k_scale", ref.rotate(host(k), cos, sin, inter)), ("V", "v_scale", host(v))):
        code, byte = bytes_of(getattr(c, pool)), bytes_of(getattr(c, scale))
        for b in range(B):
            for h in range(Hkv):
                at = np.arange(3, 3 + T) if not table else c.table_h[layer, b, h, 3:3 + T]
                written[layer, b, h, at] = True
                touched[layer, b, h, at // block] = True
                e = byte[layer, b, h, at // block].astype(int)
                x = rows[b, :, h]
                slack = 2.0 ** -21 * 2 * np.abs(x).max(-1) if pool == "K" else np.zeros(T)
                top = np.abs(x).max(-1)
                if block == 1:
                    assert ((e >= 127 + lo) & (e <= 127 + hi)).all()
                    assert ((448 * 2.0 ** (e - 127) >= top - slack) | (e == 127 + hi)).all()
                    assert ((448 * 2.0 ** (e - 128) < top + slack) | (e == 127 + lo)).all()
                else:
                    assert (e == before[2 if pool == "K" else 3][layer, b, h, at // block]).all()
                p = ref8.power(e, dtype)[:, None]
                got = ref8.CODES[code[layer, b, h, at]] * p
                if pool == "V":  # not rotated: the code is known
                    assert (code[layer, b, h, at] == ref8.encode(x / p)).all()
                held = np.clip(x, -448 * p, 448 * p)
                assert (np.abs(got - held) <= np.maximum(2.0 ** -4 * np.abs(held), 2.0 ** -10 * p) + slack[:, None] * 1.1).all()
    assert (bytes_of(c.K)[~written] == before[0][~written]).all() and (bytes_of(c.V)[~written] == before[1][~written]).all()
    assert (bytes_of(c.k_scale)[~touched] == before[2][~touched]).all() and (bytes_of(c.v_scale)[~touched] == before[3][~touched]).all()
    w = gpu(written)
    assert t.equal(c.acc[~w], acc0[~w]) and bool((c.acc[w] == 0).all())


def test_append_rows_that_are_not_finite(si):
    """A row with an infinity or NaN stands for NaN, with codes of 0; its neighbours are as they are."""
    t = torch()
    c = Cache8(si, 12, [0], 4, 2, 64, "bf16", acc=False)
    x = c.rng.standard_normal((1, 4, 2, 64))
    x[0, 1, 0, 5], x[0, 2, 1, 63] = np.inf, np.nan
    k = gpu(x, t.bfloat16)
    si.si_kv_append(c.kv, si.si_rope_create(64), None, k, k, t.zeros(1, 4, 1, dtype=t.int32, device="cuda"), None)
    for pool in ("K", "V"):
        v, code = c.values(pool), bytes_of(getattr(c, pool))
        for node in range(4):
            for h in range(2):
                slot = c.table_h[0, 0, h, node]
                odd = (node, h) in ((1, 0), (2, 1))
                assert np.isnan(v[0, h, slot]).all() == odd and (not odd or (code[0, 0, h, slot] == 0).all())


def test_append_with_given_scales_saturates(si):
    t = torch()
    c = Cache8(si, 13, [0], 3, 1, 32, "fp16", block=1 << 10)
    c.k_scale.fill_(127 - 8)
    c.v_scale.fill_(0)  # below fp16's least: taken as 2^-15
    x = np.array([0.5, 1.75, 1.76, 7.0, -60000.0, 1e-7, -0.0, 2.0 ** -8] * 4)
    k = gpu(np.broadcast_to(x, (1, 3, 1, 32)), t.float16).contiguous()
    si.si_kv_append(c.kv, si.si_rope_create(32, inv_freq=[0.0] * 8), None, k, k, t.zeros(1, 3, 1, dtype=t.int32, device="cuda"), None)
    xs = host(k)[0, 0, 0]
    for pool, p in (("K", 2.0 ** -8), ("V", 2.0 ** -15)):
        for node in range(3):
            got = bytes_of(getattr(c, pool))[0, 0, 0, c.table_h[0, 0, 0, node]]
            assert (ref8.CODES[got] == ref8.CODES[ref8.encode(xs / p)]).all()  # a turn of 0 may give 0 for -0
    assert bool((c.k_scale == 127 - 8).all()) and bool((c.v_scale == 0).all())


def test_append_out_of_bounds_is_refused(si):
    t = torch()
    c = Cache8(si, 14, [2, 2], 2, 2, 64, "bf16")
    c.lens.copy_(gpu(np.array([[2, 3]], np.int32)))  # sequence 1 has one free entry for two tokens
    c.table[0, 0, 1, 2] = 1 << 28
    K0, s0 = bytes_of(c.K).copy(), bytes_of(c.k_scale).copy()
    k = gpu(c.rng.standard_normal((2, 2, 2, 64)), t.bfloat16)
    si.si_kv_append(c.kv, si.si_rope_create(64), None, k, k, t.zeros(2, 2, 1, dtype=t.int32, device="cuda"), None)
    assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE
    same = (bytes_of(c.K) == K0).all(-1)
    assert same[0, 1].all() and (bytes_of(c.k_scale) == s0)[0, 1].all()
    assert (~same[0, 0, 0]).sum() == 2 and (~same[0, 0, 1]).sum() == 1


# ---------------------------------------------------------------- attention

CASES = [
    # lens, T, Hq, Hkv, D, dtype, table, mask, block
    ([0], 1, 1, 1, 64, "bf16", True, "none", 1),
    ([1], 1, 4, 2, 128, "fp16", False, "none", 1),
    ([62], 1, 8, 2, 64, "bf16", True, "tree", 1),
    ([63], 1, 8, 2, 64, "bf16", True, "none", 2),
    ([64], 1, 3, 3, 64, "fp16", True, "none", 1),
    ([1000], 1, 16, 2, 128, "bf16", True, "none", 1),
    ([5000], 1, 8, 1, 128, "fp16", False, "none", 64),
    ([130, 0, 700], 5, 6, 2, 128, "bf16", True, "tree", 1),
    ([60, 61, 127], 7, 9, 3, 96, "fp16", True, "tree", 1),
    ([33, 500], 16, 8, 4, 80, "bf16", True, "pad", 16),
    ([100, 3], 64, 4, 1, 128, "fp16", True, "pad", 1),
    ([2000], 33, 14, 2, 128, "bf16", True, "tree", 1),
    ([90, 700], 64, 8, 1, 64, "bf16", False, "none", 1 << 20),
    ([300], 3, 10, 2, 256, "bf16", True, "tree", 1),
    ([700], 1, 10, 2, 256, "fp16", True, "tree", 1),
    ([65, 64], 20, 8, 2, 256, "fp16", True, "pad", 1),
    ([40], 2, 2, 1, 16, "bf16", True, "tree", 1),
    ([17] * 30, 2, 4, 2, 64, "fp16", True, "tree", 1),
    ([3000, 1], 64, 16, 2, 128, "bf16", True, "pad", 8),
    ([0, 63, 64, 128], 9, 8, 2, 128, "bf16", True, "tree", 1),
    ([4000], 40, 5, 1, 64, "fp16", True, "pad", 1),
    ([1500], 17, 3, 3, 128, "fp16", False, "tree", 1),
    ([5, 70] * 100, 1, 4, 2, 64, "bf16", True, "none", 1),       # more lists than CTAs
    ([3, 130] * 100, 5, 8, 2, 64, "fp16", True, "pad", 4),
    ([9000, 1, 64, 7000, 20], 40, 8, 2, 128, "bf16", False, "tree", 1),
    ([500], 8, 1, 1, 112, "bf16", True, "tree", 1),              # eight rows a key
    ([500], 9, 1, 1, 112, "fp16", True, "tree", 1),              # nine
    ([900, 10], 16, 4, 4, 128, "fp16", True, "pad", 1),          # sixteen
    ([2, 40, 0, 129] * 200, 1, 2, 1, 128, "bf16", True, "none", 1),   # 800 sequences: the plan beside the ring
    ([2, 40] * 450, 20, 1, 1, 128, "fp16", True, "tree", 1),
    ([3, 70, 1] * 300, 2, 2, 1, 256, "bf16", True, "tree", 32),
    ([150], 4, 64, 1, 256, "fp16", True, "tree", 1),             # 256 rows a key in blocks of 16
    ([70, 300], 64, 32, 1, 64, "bf16", True, "tree", 1),         # 2048
    ([20000], 1, 8, 1, 128, "bf16", True, "none", 1),            # more parts than are joined at once
    ([12000, 5], 2, 8, 1, 256, "fp16", False, "tree", 16),
    ([30000], 1, 3, 1, 64, "fp16", True, "none", 1),
]


@pytest.mark.parametrize("lens,T,Hq,Hkv,D,dtype,table,mask,block", CASES)
def test_attention(si, lens, T, Hq, Hkv, D, dtype, table, mask, block):
    c = Cache8(si, 21, lens, T, Hkv, D, dtype, block=block, table=table, L=2, layer=1)
    q, words, mask_t = make_rows(c, T, Hq, D, dtype, mask)
    c.hide(words)
    for b in range(len(lens)):
        for node in range(T):
            if not any(int(w) >> node & 1 for w in words[b]):
                q[b, node] = float("nan")
    out, lse = Guarded(q.shape, q.dtype), Guarded(q.shape[:3], torch().float32)
    scale = 0.7 / math.sqrt(D)
    si.si_tree_attention(c.kv, q, out.t, mask=mask_t, lse=lse.t, scale=scale, layer=1)
    out.check(), lse.check()
    qz = torch().nan_to_num(q.float()).to(q.dtype)
    check(c, qz, out.t, lse.t, words, scale, dtype)
    again = torch().empty_like(q)
    si.si_tree_attention(c.kv, q, again, mask=mask_t, scale=scale, layer=1)
    assert torch().equal(again, out.t)  # no lse asked for, and the same bits


@pytest.mark.parametrize("T,Hq,Hkv,D,dtype", [(1, 4, 2, 128, "bf16"), (3, 8, 2, 64, "fp16"), (16, 4, 4, 128, "fp16"),
                                              (12, 16, 2, 128, "bf16"), (2, 2, 1, 256, "bf16"), (40, 4, 1, 64, "fp16")])
def test_attention_scales_far_apart(si, T, Hq, Hkv, D, dtype):
    """Values whose scales lie up to the type's whole range apart; keys that grow along the list."""
    c = Cache8(si, 22, [700, 90], T, Hkv, D, dtype, spread=2.0)
    lo, hi = ref8.LIMITS[dtype]
    span = (lo + 127, hi + 120) if dtype == "fp16" else (127 - 60, 127 + 60)
    c.v_scale.copy_(gpu(c.rng.integers(*span, c.v_scale.shape).astype(np.uint8)))
    q, words, mask = make_rows(c, T, Hq, D, dtype, "tree")
    out, lse = torch().empty_like(q), torch().empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, out, mask=mask, lse=lse, scale=0.5 / math.sqrt(D))
    check(c, q, out, lse, words, 0.5 / math.sqrt(D), dtype)


@pytest.mark.parametrize("T,Hq,Hkv,D,dtype", [(1, 4, 2, 128, "bf16"), (8, 4, 2, 128, "fp16"), (20, 8, 2, 64, "bf16"), (3, 8, 2, 256, "bf16")])
def test_attention_queries_of_any_size(si, T, Hq, Hkv, D, dtype):
    """Query rows from the type's small to its large numbers beside one another, and rows of zeros."""
    c = Cache8(si, 23, [300], T, Hkv, D, dtype)
    q, words, mask = make_rows(c, T, Hq, D, dtype, "tree")
    size = 2.0 ** c.rng.integers(-20, 6, (1, T, Hq, 1)) if dtype == "fp16" else 2.0 ** c.rng.integers(-100, 6, (1, T, Hq, 1))
    q = (q.double() * gpu(size)).to(q.dtype)
    q[0, 0, -1] = 0.0
    q[0, -1, 0, ::3] *= 2.0 ** -12  # a row whose elements lie far apart
    out, lse = torch().empty_like(q), torch().empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, out, mask=mask, lse=lse, scale=0.5 / math.sqrt(D))
    check(c, q, out, lse, words, 0.5 / math.sqrt(D), dtype)
    if dtype == "bf16":  # 2^40 times, with keys 2^-40 as large: the same scores
        before = out.clone()
        c.k_scale.copy_(torch().where(c.k_scale == 255, c.k_scale, c.k_scale - 40))
        si.si_tree_attention(c.kv, q * 2.0 ** 40, out, mask=mask, scale=0.5 / math.sqrt(D))
        assert torch().equal(out, before)


@pytest.mark.parametrize("T,Hq,Hkv,D,dtype,block", [(4, 2, 1, 64, "bf16", 1), (4, 8, 2, 128, "fp16", 1), (16, 8, 2, 128, "bf16", 1),
                                                    (40, 8, 2, 64, "fp16", 1), (6, 2, 2, 256, "bf16", 1),
                                                    (4, 2, 1, 64, "bf16", 64), (40, 8, 2, 128, "bf16", 64), (6, 4, 2, 256, "fp16", 64)])
def test_nan_of_a_node_reaches_only_those_that_see_it(si, T, Hq, Hkv, D, dtype, block):
    """A node's row of NaN (its scale's, or with shared scales its codes'), as key or as value; siblings do not see it."""
    t = torch()
    for n in (100, 64 - T // 2, 0):
        for part in ("K", "V"):
            c = Cache8(si, 24, [n], T, Hkv, D, dtype, block=block)
            words = np.array([[1 << i | 1 for i in range(T)]], np.uint64)  # all children of node 0
            q = gpu(c.rng.standard_normal((1, T, Hq, D)), tdtype(dtype))
            run = lambda: si.si_tree_attention(c.kv, q, t.empty_like(q), mask=gpu(words.view(np.int64)))  # noqa: E731
            clean = run()
            node = T - 1
            for h in range(Hkv):
                slot = int(c.table_h[0, 0, h, n + node])
                if block == 1:
                    getattr(c, part.lower() + "_scale")[0, 0, h, slot] = 255
                    getattr(c, part).view(t.uint8)[0, 0, h, slot] = 0
                else:
                    getattr(c, part).view(t.uint8)[0, 0, h, slot, 7] = 0x7F
            got = run()
            assert t.equal(got[0, :node], clean[0, :node])
            nan = got[0, node].isnan()
            assert bool(nan.all()) if block == 1 or part == "K" else bool(nan[:, 7].all()) and int(nan.sum()) == Hq


def test_attention_rows_that_see_nothing(si):
    """Lengths out of bounds and padding give zeros and -inf, and set the error; the other sequences are served."""
    t = torch()
    for T, Hq in ((2, 4), (64, 8)):
        c = Cache8(si, 25, [100, 100, 100], T, 2, 64, "bf16")
        c.lens.copy_(gpu(np.array([[100, 101, -1]], np.int32)))
        q = gpu(c.rng.standard_normal((3, T, Hq, 64)), t.bfloat16)
        out, lse = t.full_like(q, 7.0), t.zeros(3, T, Hq, device="cuda")
        si.si_tree_attention(c.kv, q, out, lse=lse)
        assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE
        assert bool((out[1:] == 0).all()) and bool(lse[1:].isneginf().all()) and bool(lse[0].isfinite().all())
        words = t.zeros(3, T, dtype=t.int64, device="cuda")
        si.si_tree_attention(c.kv, q, out, mask=words, lse=lse)
        assert bool((out == 0).all()) and bool(lse.isneginf().all())
        si.si_device_error(clear=True)


@pytest.mark.parametrize("T,Hq,D", [(2, 4, 128), (20, 8, 64), (3, 2, 256)])
def test_strided_operands(si, T, Hq, D):
    """Pools, scales, tables, weights and queries that are slices of larger arrays give the bits of contiguous ones."""
    t = torch()
    c = Cache8(si, 30, [150, 64], T, 2, D, "bf16", slack=5)
    q, words, mask = make_rows(c, T, Hq, D, "bf16", "tree")
    want, lse, acc = t.empty_like(q), t.empty(q.shape[:3], device="cuda"), c.acc.clone()
    si.si_tree_attention(c.kv, q, want, mask=mask, lse=lse)
    si.si_kv_accumulate(c.kv, q, lse, mask=mask)

    def within(a, pads):
        """The same array as a slice of a larger one full of other numbers; the last dimension stays whole."""
        big = t.full([n + p for n, p in zip(a.shape, pads)], 0x7F if a.element_size() == 1 else 7, device="cuda",
                     dtype=t.uint8 if a.element_size() == 1 else a.dtype)
        cut = tuple(slice(p // 2 // 16 * 16 if i == len(pads) - 1 else p // 2, p // 2 // 16 * 16 + n if i == len(pads) - 1 else p // 2 + n)
                    for i, (n, p) in enumerate(zip(a.shape, pads)))
        part = big[cut]
        part.copy_(a.view(t.uint8) if a.element_size() == 1 else a)
        return part.view(a.dtype)

    K, V = within(c.K, (0, 1, 2, 3, 32)), within(c.V, (0, 2, 1, 5, 64))
    ks, vs = within(c.k_scale, (1, 0, 1, 32)), within(c.v_scale, (0, 1, 1, 64))
    table, acc2 = within(c.table, (1, 1, 1, 0)), within(acc, (1, 0, 1, 32))
    kv = si.si_kv_create(K, V, table, c.lens, acc2, k_scale=ks, v_scale=vs)
    q2, got, lse2 = within(q, (1, 2, 1, 32)), t.empty_like(q), t.empty_like(lse)
    si.si_tree_attention(kv, q2, got, mask=mask, lse=lse2)
    si.si_kv_accumulate(kv, q2, lse2, mask=mask)
    assert t.equal(got, want) and t.equal(lse2, lse) and t.equal(acc2, c.acc)


def test_attention_slot_outside_the_pool(si):
    t = torch()
    for T, Hq in ((1, 4), (40, 4)):
        c = Cache8(si, 26, [200], T, 2, 64, "bf16")
        c.table[0, 0, 0, 70] = 1 << 30
        c.table[0, 0, 1, 3] = -5
        q = gpu(c.rng.standard_normal((1, T, Hq, 64)), t.bfloat16)
        si.si_tree_attention(c.kv, q, t.empty_like(q))
        assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE


@pytest.mark.parametrize("T,Hq,Hkv,D", [(64, 32, 8, 128), (16, 16, 4, 128), (4, 4, 2, 64), (1, 8, 2, 128)])
def test_attention_back_to_back(si, T, Hq, Hkv, D):
    """Launches that overlap their neighbours' ends, by the hundred, eager and from a graph: every one has the same bits."""
    t = torch()
    c = Cache8(si, 27, [3000, 1900, 700], T, Hkv, D, "bf16")
    q, words, mask = make_rows(c, T, Hq, D, "bf16", "tree" if T > 1 else "none")
    want, outs = t.empty_like(q), [t.zeros_like(q) for _ in range(100)]
    si.si_tree_attention(c.kv, q, want, mask=mask)
    for o in outs:
        si.si_tree_attention(c.kv, q, o, mask=mask)
    assert all(t.equal(o, want) for o in outs)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        for o in outs:
            si.si_tree_attention(c.kv, q, o, mask=mask)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        assert all(t.equal(o, want) for o in outs)
    assert si.si_device_error() == 0


def test_pools_past_32_bits(si):
    """Slots whose bytes lie past 2^32, scales of single slots and strided pools."""
    t = torch()
    n_slots, D, n = 30_000_000, 128, 300
    wide = t.empty(1, 1, 2, n_slots, D + 32, dtype=t.uint8, device="cuda")  # 4.8 GB a head
    K = wide[..., :D].view(t.float8_e4m3fn)
    byte = t.empty(1, 1, 2, n_slots, dtype=t.uint8, device="cuda")
    rng = np.random.default_rng(28)
    for T, Hq in ((1, 4), (24, 4)):
        table_h = np.stack([np.sort(rng.choice(n_slots, n + T, False))[::-1] for _ in range(2)])[None, None].astype(np.int32)
        code, e = rng.integers(0, 0x70, (2, n + T, D)).astype(np.uint8), rng.integers(115, 122, (2, n + T)).astype(np.uint8)
        for h in range(2):
            at = gpu(table_h[0, 0, h].astype(np.int64))
            wide[0, 0, h, at, :D] = gpu(code[h])
            byte[0, 0, h, at] = gpu(e[h])
        acc = t.zeros(1, 1, 2, n_slots, device="cuda")
        kv = si.si_kv_create(K, K, gpu(table_h), gpu(np.array([[n]], np.int32)), acc, k_scale=byte, v_scale=byte)
        q = gpu(rng.standard_normal((1, T, Hq, D)) * 0.02, t.bfloat16)
        out, lse = t.empty_like(q), t.empty(1, T, Hq, device="cuda")
        si.si_tree_attention(kv, q, out, lse=lse)
        x = (ref8.CODES[code] * ref8.power(e, "bf16")[..., None])[None]
        want, lse_w, mag = ref.attend(host(q), x, x, None, [n], ref.chain(1, T), D ** -0.5)
        assert np.abs(host(lse) - lse_w).max() <= 1e-4
        assert (np.abs(host(out) - want) <= 2.0 ** -7 * mag + 1e-3 * mag).all()
        si.si_kv_accumulate(kv, q, lse)
        got = np.stack([acc[0, 0, h, gpu(table_h[0, 0, h].astype(np.int64))].double().cpu().numpy() for h in range(2)])
        w = ref.weigh(host(q), x, None, [n], ref.chain(1, T), None, lse_w, np.zeros((1, 2, n + T)), D ** -0.5)[0]
        assert np.abs(got - w).max() <= 1e-3
        assert si.si_device_error() == 0
        kv.close()
        del acc


# ------------------------------------------------------------------ weights

WEIGH = [
    # lens, T, Hq, Hkv, D, dtype, table, mask, rows, block
    ([0], 1, 2, 1, 64, "bf16", True, "none", None, 1),
    ([100, 63], 1, 8, 2, 64, "fp16", True, "none", None, 1),
    ([1000, 5, 64], 5, 6, 2, 128, "bf16", True, "tree", [0b10011, 0, 0b1], 1),
    ([300, 65], 20, 8, 2, 96, "fp16", True, "pad", None, 16),
    ([500], 64, 16, 2, 128, "bf16", False, "pad", None, 1),     # 512 rows a key
    ([200], 3, 4, 2, 256, "bf16", True, "tree", [0b110], 1 << 12),
    ([70], 40, 10, 1, 256, "fp16", True, "tree", None, 1),
    ([30, 31], 2, 2, 2, 16, "bf16", True, "tree", None, 1),
    ([5, 70] * 60, 3, 4, 2, 80, "bf16", True, "tree", None, 1),
    ([2, 40, 0, 129] * 200, 1, 2, 1, 128, "bf16", True, "none", None, 1),
    ([150], 4, 64, 1, 128, "fp16", True, "tree", [0b1010], 1),
]


@pytest.mark.parametrize("lens,T,Hq,Hkv,D,dtype,table,mask,rows,block", WEIGH)
def test_weights(si, lens, T, Hq, Hkv, D, dtype, table, mask, rows, block):
    t = torch()
    c = Cache8(si, 31, lens, T, Hkv, D, dtype, block=block, table=table, L=2, layer=1)
    q, words, mask_t = make_rows(c, T, Hq, D, dtype, mask)
    c.hide(words)
    for b in range(len(lens)):
        for node in range(T):
            if words[b, node] == 0:
                q[b, node] = float("nan")
    scale = 0.7 / math.sqrt(D)
    out, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
    si.si_tree_attention(c.kv, q, out, mask=mask_t, lse=lse, scale=scale, layer=1)
    rows_h = None if rows is None else np.array(rows, np.uint64)
    dst = t.full_like(c.acc[1], -3.0)
    si.si_kv_accumulate(c.kv, q, lse, mask=mask_t, rows=None if rows is None else gpu(rows_h.view(np.int64)), scale=scale, acc_out=dst, layer=1)
    K, _, tab = c.args()
    qz = np.nan_to_num(host(q))
    want = ref.weigh(qz, np.nan_to_num(K), tab, c.lens_h, words, rows_h, host(lse), host(c.acc[1]), scale)
    e = score_error(qz, K, D, scale) + 2.0 ** -19
    G = Hq // Hkv
    for b, n in enumerate(lens):
        for h in range(Hkv):
            at = np.arange(n + T) if tab is None else tab[b, h, :n + T]
            got, w = host(dst[b, h])[at], want[b, h, at]
            assert (np.abs(got - w) <= (np.expm1(e) + T * G * 2.0 ** -23) * np.abs(w) + 2.0 ** -23 * (1 + np.abs(w))).all()
            rest = np.setdiff1d(np.arange(dst.shape[2]), at)
            assert (host(dst[b, h])[rest] == -3.0).all()
    again = t.full_like(dst, -3.0)
    si.si_kv_accumulate(c.kv, q, lse, mask=mask_t, rows=None if rows is None else gpu(rows_h.view(np.int64)), scale=scale, acc_out=again, layer=1)
    assert t.equal(again, dst)
    before = c.acc.clone()
    si.si_kv_accumulate(c.kv, q, lse, mask=mask_t, rows=None if rows is None else gpu(rows_h.view(np.int64)), scale=scale, layer=1)
    listed = dst != -3.0
    assert t.equal(c.acc[1][listed], dst[listed]) and t.equal(c.acc[1][~listed], before[1][~listed]) and t.equal(c.acc[0], before[0])


def test_weights_of_nan_and_out_of_bounds(si):
    """A key of NaN that a row does not see gives it nothing; bad lengths and slots are reported and left alone."""
    t = torch()
    c = Cache8(si, 32, [40, 40], 3, 1, 64, "bf16")
    words = np.array([[1, 3, 5]] * 2, np.uint64)
    slot = int(c.table_h[0, 0, 0, 42])
    c.k_scale[0, 0, 0, slot] = 255
    c.table[0, 0, 0, 7] = 1 << 25
    c.lens.copy_(gpu(np.array([[40, 41]], np.int32)))
    q = gpu(c.rng.standard_normal((2, 3, 2, 64)), t.bfloat16)
    lse = t.full((2, 3, 2), 3.0, device="cuda")
    before = c.acc.clone()
    si.si_kv_accumulate(c.kv, q, lse, mask=gpu(words.view(np.int64)), rows=gpu(np.array([3, 3], np.int64)))
    assert si.si_device_error(clear=True) == si.SI_DEVERR_CACHE
    assert t.equal(c.acc[0, 1], before[0, 1])
    assert bool(c.acc.isfinite().all()) and float(c.acc[0, 0, 0, slot]) == float(before[0, 0, 0, slot])


# --------------------------------------------------------------- as they are used

@pytest.mark.parametrize("dtype,block", [("bf16", 1), ("fp16", 1), ("bf16", 1 << 12)])
def test_a_run_of_steps(si, dtype, block):
    """Prompt, drafted trees, weights and eviction over many steps, next to a cache in 16 bits that holds what the codes
    stand for: the attention's outputs agree within both kernels' bounds, the lists stay the same permutations."""
    t = torch()
    L, B, Hkv, G, D, cap, T = 2, 2, 2, 4, 64, 200, 6
    td = tdtype(dtype)
    rng = np.random.default_rng(41)
    K, V = (t.zeros(L, B, Hkv, cap, D, device="cuda").to(t.float8_e4m3fn) for _ in range(2))
    ks, vs = (t.full((L, B, Hkv, -(-cap // block)), 120, dtype=t.uint8, device="cuda") for _ in range(2))
    table = t.arange(cap, dtype=t.int32, device="cuda").expand(L, B, Hkv, cap).contiguous()
    lens, acc = t.zeros(L, B, dtype=t.int32, device="cuda"), t.zeros(L, B, Hkv, cap, device="cuda")
    kv = si.si_kv_create(K, V, table, lens, acc, k_scale=ks, v_scale=vs, block=block, dtype=td)
    rope = si.si_rope_create(D)
    done = 0
    for step in range(30):
        n = 60 if step == 0 else T
        words = ref.chain(B, n) if step == 0 else ref.trees(rng, B, n)
        for layer in range(L):
            qkv = gpu(rng.standard_normal((B, n, (G + 2) * Hkv, D)), td)
            q = t.empty(B, n, G * Hkv, D, dtype=td, device="cuda")
            pos = gpu(np.broadcast_to((done + np.arange(n))[None, :, None], (B, n, 1)).astype(np.int32))
            si.si_kv_append(kv, rope, qkv[:, :, :G * Hkv], qkv[:, :, G * Hkv:(G + 1) * Hkv], qkv[:, :, (G + 1) * Hkv:], pos, q, layer=layer)
            out, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
            si.si_tree_attention(kv, q, out, mask=gpu(words.view(np.int64)), lse=lse, layer=layer)
            si.si_kv_accumulate(kv, q, lse, mask=gpu(words.view(np.int64)), layer=layer)
            x, y = (ref8.decode(bytes_of(p[layer]), bytes_of(e[layer]), dtype, block) for p, e in ((K, ks), (V, vs)))
            lens_h = lens[layer].cpu().numpy()
            want, lse_w, mag = ref.attend(host(q), x, y, table[layer].cpu().numpy(), lens_h, words, D ** -0.5)
            e = score_error(host(q), x, D, D ** -0.5) + 2.0 ** -19
            assert (np.abs(host(out) - want) <= ref.U[dtype] * (mag + np.abs(want)) + 2 * e * mag + 2.0 ** -24).all(), step
            assert np.abs(host(lse) - lse_w).max() <= e + 2.0 ** -20 * 10
        path = np.zeros((B, n), np.int32)
        count = np.full(B, n if step == 0 else 2, np.int32)
        path[:, :] = np.arange(n)
        if step:
            si.si_kv_evict(kv, n, 90, sinks=2, recent=16, path=gpu(path), n_path=gpu(count))
        else:
            si.si_kv_evict(kv, n, 90, sinks=2, recent=16)
        done += int(count[0])
        assert (np.sort(table.cpu().numpy(), -1) == np.arange(cap)).all()
        assert (lens.cpu().numpy() == min(done if done <= 90 else 90, 90)).all()
    assert si.si_device_error() == 0


def test_a_step_in_a_graph_on_another_stream(si):
    """Append, attention, weights and eviction captured once and replayed, on a stream of its own."""
    t = torch()
    lens, T, Hkv, Hq, D = [50, 20], 3, 2, 8, 64
    caches = [Cache8(si, 42, lens, T, Hkv, D, "bf16", slack=40) for _ in range(2)]
    rope = si.si_rope_create(D)
    rng = caches[0].rng
    qkv = gpu(rng.standard_normal((2, T, Hq + 2 * Hkv, D)), t.bfloat16)
    pos = t.zeros(2, T, 1, dtype=t.int32, device="cuda")

    def step(c, q, out, lse):
        si.si_kv_append(c.kv, rope, qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:], pos, q)
        si.si_tree_attention(c.kv, q, out, lse=lse)
        si.si_kv_accumulate(c.kv, q, lse)
        si.si_kv_evict(c.kv, T, 55, sinks=2, recent=8)

    bufs = [(t.empty(2, T, Hq, D, dtype=t.bfloat16, device="cuda"), t.empty(2, T, Hq, D, dtype=t.bfloat16, device="cuda"),
             t.empty(2, T, Hq, device="cuda")) for _ in range(2)]
    for _ in range(4):
        step(caches[0], *bufs[0])
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(caches[1], *bufs[1])
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            step(caches[1], *bufs[1])
        for _ in range(3):
            g.replay()
    side.synchronize()
    for a in ("K", "V", "k_scale", "v_scale", "table", "lens"):
        assert (bytes_of(getattr(caches[0], a)) == bytes_of(getattr(caches[1], a))).all(), a
    assert t.equal(caches[0].acc, caches[1].acc) and all(t.equal(x, y) for x, y in zip(*bufs))
