"""Cases of the key/value cache operators: rotary append, tree attention, attention-weight accumulation and eviction.

A decode step with drafted tokens runs, per layer, `si_kv_append` (rotate the new queries and keys, write keys and
values into free slots), `si_tree_attention` (every drafted token over the cached keys and its own ancestors),
`si_kv_accumulate` (the weight each cached key received from the accepted tokens) and, once a step, `si_kv_evict`
(accept a path of the tree, drop the keys with the least accumulated weight). A cache is K and V
[layer][sequence][head][slot][D], a slot table [layer][sequence][head][entry] whose first len[layer][sequence] entries
are the live keys in insertion order (the rest are free slots), and the accumulated weights per slot.

Each case names its operator in "op". Where `own` is false, `run` computes it with elementary torch operations;
where it is true, it calls the framework.
"""
import math
import types

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ROPE_BASE = 500000.0


def listed():
    return [
        # one new token of one sequence: the smallest append, all latency
        dict(name="append-token", op="append", B=1, T=1, Hq=32, Hkv=8, D=64, axes=1, interleaved=False, dtype="bf16", far=4096),
        # drafted trees of a batch, at far text positions
        dict(name="append-tree", op="append", B=8, T=33, Hq=32, Hkv=8, D=128, axes=1, interleaved=True, dtype="fp16", far=1000000),
        # a prompt with images: three axes
        dict(name="append-prompt", op="append", B=1, T=8192, Hq=32, Hkv=8, D=128, axes=3, interleaved=False, dtype="bf16", far=16384),
        # one token over a short chat, an evicted cache
        dict(name="attend-token", op="attend", B=1, T=1, Hq=32, Hkv=8, D=64, len=1000, ragged=False, order="evicted", dtype="bf16"),
        # a drafted tree of 16 over a batch of unequal contexts
        dict(name="attend-tree", op="attend", B=6, T=16, Hq=16, Hkv=2, D=128, len=9001, ragged=True, order="evicted", dtype="bf16"),
        # one token over a long document that never evicted
        dict(name="attend-long", op="attend", B=1, T=1, Hq=32, Hkv=8, D=128, len=131071, ragged=False, order="fresh", dtype="bf16"),
        # wide trees of a batch: the most rows a key meets
        dict(name="attend-wide", op="attend", B=8, T=64, Hq=32, Hkv=8, D=128, len=8192, ragged=True, order="evicted", dtype="fp16"),
        # weights of one token's attention
        dict(name="weigh-token", op="weigh", B=1, T=1, n_rows=1, Hq=32, Hkv=8, D=64, len=4095, ragged=False, order="evicted", dtype="bf16"),
        # weights of the accepted tokens of a batch of trees
        dict(name="weigh-tree", op="weigh", B=8, T=16, n_rows=4, Hq=32, Hkv=8, D=128, len=16384, ragged=True, order="evicted", dtype="bf16"),
        # one layer, one token over a small budget
        dict(name="evict-token", op="evict", L=1, B=1, Hkv=8, T=1, n_path=1, len=1024, ragged=False, budget=1024, sinks=4, recent=128),
        # a whole model's step after a drafted tree
        dict(name="evict-step", op="evict", L=28, B=4, Hkv=8, T=16, n_path=5, len=4096, ragged=False, budget=4096, sinks=4, recent=512),
        # long prompts cut down to a budget
        dict(name="evict-prompt", op="evict", L=2, B=4, Hkv=8, T=1, n_path=1, len=100000, ragged=True, budget=16384, sinks=16, recent=1024),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of its range."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weigh", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        B = rng.choice([1, 2, 3, 8])
        T = _log(rng, 1, 8192 // B)
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=min(D, 128), axes=rng.choice([1, 2, 3]), interleaved=rng.choice([False, True]),
                    dtype=dtype, far=_log(rng, 100, 2000000))
    if op == "evict":
        L, B = rng.choice([1, 2, 16]), rng.choice([1, 2, 5])
        T = rng.choice([1, 1, 5, 16, 64])
        n = _log(rng, 40, 800000 // (L * B))
        n = min(n, 120000)
        budget = max(8, int(n * rng.uniform(0.1, 1.05)))
        return dict(op=op, L=L, B=B, Hkv=Hkv, T=T, n_path=rng.randint(1, min(T, 8)), len=n, ragged=rng.choice([False, True]), budget=budget,
                    sinks=rng.choice([0, 4]), recent=budget // rng.choice([2, 8, 64]))
    B = rng.choice([1, 1, 2, 4, 7])
    T = rng.choice([1, 1, 2, 5, 8, 16, 31, 64])
    top = min(131072, 2 ** 27 // (B * Hkv * D), 2 ** 33 // (B * Hkv * G * T * D))  # at most the long document's keys, the wide tree's products
    n = _log(rng, 1, top)
    case = dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, len=n, ragged=rng.choice([False, True]), order=rng.choice(["evicted", "fresh"]),
                dtype=dtype)
    if op == "weigh":
        case["n_rows"] = rng.randint(1, min(T, 8))
    return case


def _lens(case):
    """Live entries of each sequence: all `len`, or falling from it in equal steps."""
    B = case["B"]
    return [case["len"] * (B - b) // B if case.get("ragged") else case["len"] for b in range(B)]


def _nodes(case):
    """Drafted nodes of each sequence (the rest of T is padding)."""
    return [max(1, case["T"] - (b % 3) * (case["T"] // 8)) if case.get("ragged") else case["T"] for b in range(case["B"])]


def _tree(case, seed):
    """Ancestor words int64 [B][T]: bit j of word t says that node t sees node j; a padding node's word is 0."""
    rng = np.random.RandomState(seed % 2 ** 31)
    words = np.zeros((case["B"], case["T"]), np.uint64)
    for b, nodes in enumerate(_nodes(case)):
        for t in range(nodes):
            parent = rng.randint(max(-1, t - 6), t) if t else -1
            words[b, t] = np.uint64(1 << t) | (words[b, parent] if parent >= 0 else np.uint64(0))
    return words.view(np.int64)


def _table(gen, lead, entries, order):
    """A slot table: slots in order (a cache that never evicted) or in the mixed order that many evictions leave."""
    if order == "fresh":
        return torch.arange(entries, dtype=torch.int32, device="cuda").expand(*lead, entries).contiguous()
    return torch.rand(*lead, entries, generator=gen, device="cuda").argsort(-1).to(torch.int32)


def _sections(D, axes):
    """Rotary pairs of each axis: D / 2 in all."""
    half = D // 2
    first = half - (axes - 1) * (half // (axes + 1))
    return [first] + [half // (axes + 1)] * (axes - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = types.SimpleNamespace(op=case["op"])
    rnd = lambda *shape, dtype=torch.float32: torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    B, T, Hkv = case["B"], case["T"], case["Hkv"]
    if s.op == "evict":
        L, cap, n = case["L"], case["len"] + case["T"], case["n_path"]
        s.table = _table(gen, (L, B, Hkv), cap, "evicted")
        s.lens = torch.tensor([_lens(case)] * L, dtype=torch.int32, device="cuda")
        # weights fall off over a few decades; young keys have little so far
        s.acc = torch.exp(2.0 * rnd(L, B, Hkv, cap))
        s.n_path = torch.tensor([min(n, 1 + (b + n) % n) for b in range(B)], dtype=torch.int32, device="cuda")
        s.path = torch.rand(B, T, generator=gen, device="cuda").argsort(-1)[:, :n].sort(-1).values.to(torch.int32)
        s.path = torch.cat([s.path, torch.zeros(B, T - n, dtype=torch.int32, device="cuda")], 1)
        s.T, s.budget, s.sinks, s.recent = T, case["budget"], case["sinks"], case["recent"]
        s.table_out, s.lens_out = torch.empty_like(s.table), torch.empty_like(s.lens)
        s.K = s.V = torch.empty(L, B, Hkv, cap, 8, dtype=torch.bfloat16, device="cuda")  # eviction moves no key
        if own:
            import activation_sparse_gb300 as si
            s.kv = si.si_kv_create(s.K, s.V, s.table, s.lens, s.acc)
        return s
    Hq, D, dtype = case["Hq"], case["D"], DTYPES[case["dtype"]]
    if s.op == "append":
        entries = T + 64
        s.K, s.V = torch.zeros(1, B, Hkv, entries, D, dtype=dtype, device="cuda"), torch.zeros(1, B, Hkv, entries, D, dtype=dtype, device="cuda")
        s.table = _table(gen, (1, B, Hkv), entries, "evicted")
        s.lens = torch.full((1, B), 7, dtype=torch.int32, device="cuda")
        s.acc = torch.ones(1, B, Hkv, entries, device="cuda")
        qkv = rnd(B, T, Hq + 2 * Hkv, D).to(dtype)  # one projection's output: q, k and v are slices of it
        s.q, s.k, s.v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s.pos = torch.randint(0, case["far"], (B, T, case["axes"]), generator=gen, device="cuda", dtype=torch.int32)
        s.sections, s.interleaved = _sections(D, case["axes"]), case["interleaved"]
        s.inv_freq = ROPE_BASE ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        s.axis = torch.tensor([a for a, n in enumerate(s.sections) for _ in range(n)], device="cuda")
        s.q_out = torch.empty(B, T, Hq, D, dtype=dtype, device="cuda")
        if own:
            import activation_sparse_gb300 as si
            s.rope = si.si_rope_create(D, base=ROPE_BASE, sections=s.sections, interleaved=s.interleaved)
            s.kv = si.si_kv_create(s.K, s.V, s.table, s.lens, s.acc)
        return s
    cap = case["len"] + T
    s.K, s.V = rnd(1, B, Hkv, cap, D, dtype=dtype), rnd(1, B, Hkv, cap, D, dtype=dtype)
    s.q = (1.5 * rnd(B, T, Hq, D)).to(dtype)
    s.table = _table(gen, (1, B, Hkv), cap, case["order"])
    s.lens = torch.tensor([_lens(case)], dtype=torch.int32, device="cuda")
    s.mask = torch.from_numpy(_tree(case, seed)).cuda()
    s.scale = 1.0 / math.sqrt(D)
    s.acc = None
    if s.op == "attend":
        s.out, s.lse = torch.empty_like(s.q), torch.empty(B, T, Hq, device="cuda")
    else:
        s.acc = torch.rand(1, B, Hkv, cap, generator=gen, device="cuda")
        s.acc_out = torch.zeros_like(s.acc)
        counted = torch.zeros(B, dtype=torch.int64)
        for b, nodes in enumerate(_nodes(case)):
            counted[b] = sum(1 << (i * nodes // case["n_rows"]) for i in range(min(nodes, case["n_rows"])))
        s.rows = counted.cuda()
        s.lse = torch.cat([_softmax(*_scores(s.q[b:b + 1], s.K[:, b:b + 1], s.table[:, b:b + 1], s.scale),
                                    _visible(s.lens[:, b:b + 1], s.mask[b:b + 1], cap))[1] for b in range(B)])
    if own:
        import activation_sparse_gb300 as si
        s.kv = si.si_kv_create(s.K, s.V, s.table, s.lens, s.acc)
    return s


# ------------------------------------------------------------------ the plain forms

def _rotate(x, cos, sin, interleaved):
    """x [B, T, H, D] with the angles' cos and sin [B, T, 1, D / 2]; rounded once, to x's type."""
    f = x.float()
    half = f.shape[-1] // 2
    a, b = (f[..., 0::2], f[..., 1::2]) if interleaved else (f[..., :half], f[..., half:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    return (torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)).to(x.dtype)


def _append(s):
    angle = s.pos.double()[..., s.axis] * s.inv_freq  # far positions: the angle needs 64 bits
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    B, T = s.pos.shape[:2]
    at = s.lens[0, :, None].long() + torch.arange(T, device="cuda")
    slot = s.table[0].gather(2, at[:, None, :].expand(-1, s.table.shape[2], -1)).long()
    rows = slot[..., None].expand(-1, -1, -1, s.K.shape[-1])
    s.K[0].scatter_(2, rows, _rotate(s.k, cos, sin, s.interleaved).transpose(1, 2))
    s.V[0].scatter_(2, rows, s.v.transpose(1, 2))
    s.acc[0].scatter_(2, slot, 0.0)
    s.q_out.copy_(_rotate(s.q, cos, sin, s.interleaved))
    return [s.q_out, s.K, s.V, s.acc]


def _visible(lens, words, entries):
    """Which list entries each drafted node sees: bool [B, T, entries]."""
    i = torch.arange(entries, device="cuda")
    j = i[None] - lens[0, :, None].long()  # the draft's own index, negative for a cached key
    T = words.shape[1]
    bit = (words[:, :, None] >> j.clamp(0, T - 1)[:, None, :]) & 1
    return ((j < 0)[:, None, :] | ((j < T)[:, None, :] & (bit != 0))) & (words != 0)[:, :, None]


def _listed(pool, table):
    """The pool's rows in list order, in 32 bits."""
    return pool[0].gather(2, table[0].long()[..., None].expand(-1, -1, -1, pool.shape[-1])).float()


def _scores(q, K, table, scale):
    """Scaled products [B, Hkv, T, G, entries] and the group size."""
    B, T, Hq, D = q.shape
    Hkv = K.shape[2]
    rows = q.float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    return ((rows @ _listed(K, table).transpose(2, 3)) * scale).view(B, Hkv, T, Hq // Hkv, -1),


def _softmax(scores, visible):
    """exp(score - max) over the visible entries with its sum, and the log-sum-exp [B, T, Hq]; a row that sees nothing has sum 0."""
    scores = scores.masked_fill(~visible[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (scores - top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    return (p, total), lse.permute(0, 2, 1, 3).flatten(2)


def _attend(s):
    B, T, Hq, D = s.q.shape
    (p, total), lse = _softmax(*_scores(s.q, s.K, s.table, s.scale), _visible(s.lens, s.mask, s.table.shape[-1]))
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = p.flatten(2, 3) @ _listed(s.V, s.table)
    s.out.copy_(o.view(B, -1, T, Hq // s.K.shape[2], D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D))
    s.lse.copy_(lse)
    return [s.out, s.lse]


def _weigh(s):
    B, T, Hq, _ = s.q.shape
    entries = s.table.shape[-1]
    (scores,) = _scores(s.q, s.K, s.table, s.scale)
    visible = _visible(s.lens, s.mask, entries) & ((s.rows[:, None] >> torch.arange(T, device="cuda")) & 1 != 0)[:, :, None]
    lse = s.lse.view(B, T, -1, scores.shape[3]).permute(0, 2, 1, 3)[..., None]
    w = (scores - lse).exp_().masked_fill_(~visible[:, None, :, None], 0.0).sum((2, 3))
    slot = s.table[0].long()
    listed_now = torch.arange(entries, device="cuda") < s.lens[0, :, None, None] + T
    s.acc_out[0].scatter_(2, slot, torch.where(listed_now, s.acc[0].gather(2, slot) + w, s.acc_out[0].gather(2, slot)))
    return [s.acc_out]


def _evict(s):
    L, B, H, cap = s.table.shape
    i = torch.arange(cap, device="cuda")
    T, n_old, n_path = s.T, s.lens.long()[:, :, None, None], s.n_path.long()[None, :, None, None]
    j = i - n_old  # [L, B, 1, cap]
    # a draft's rank in the accepted path (none: T)
    hit = (s.path[:, None, :] == torch.arange(T, device="cuda")[:, None]) & (torch.arange(T, device="cuda") < s.n_path[:, None])[:, None, :]
    rank = torch.where(hit.any(-1), hit.int().argmax(-1), T)  # [B, T]
    rank = rank[None].expand(L, -1, -1).gather(2, j[:, :, 0].clamp(0, T - 1))[:, :, None]
    live, draft = j < 0, (j >= 0) & (j < T)
    accepted = draft & (rank < T)
    # candidate order: live entries, then accepted drafts in path order
    order = torch.where(live, i, torch.where(accepted, n_old + rank, cap)).expand(L, B, H, cap)
    n = n_old + n_path
    cand = order < cap
    safe = cand & ((order < s.sinks) | (order >= n - s.recent))
    weight = s.acc.gather(3, s.table.long())
    # rank by (protected, weight) falling, ties to the lower candidate index
    by_order = order.argsort(dim=-1, stable=True)
    key = torch.where(safe, math.inf, torch.where(cand, weight, -math.inf)).gather(3, by_order)
    best = by_order.gather(3, key.argsort(dim=-1, descending=True, stable=True))
    place = torch.empty_like(best).scatter_(3, best, i.expand(L, B, H, cap).contiguous())
    kept = cand & (place < s.budget)
    group = torch.where(kept, 0, torch.where(cand, 1, torch.where(draft, 2, 3)))
    within = torch.where(cand, order, i)
    last = (group * (2 * cap) + within).argsort(-1)
    s.table_out.copy_(s.table.gather(3, last))
    s.lens_out.copy_(kept.sum(-1)[:, :, 0])
    return [s.table_out, s.lens_out]


def run(state):
    s = state
    if not own:
        return {"append": _append, "attend": _attend, "weigh": _weigh, "evict": _evict}[s.op](s)
    import activation_sparse_gb300 as si
    if s.op == "append":
        si.si_kv_append(s.kv, s.rope, s.q, s.k, s.v, s.pos, s.q_out)
        return [s.q_out, s.K, s.V, s.acc]
    if s.op == "attend":
        si.si_tree_attention(s.kv, s.q, s.out, mask=s.mask, lse=s.lse, scale=s.scale)
        return [s.out, s.lse]
    if s.op == "weigh":
        si.si_kv_accumulate(s.kv, s.q, s.lse, mask=s.mask, rows=s.rows, scale=s.scale, acc_out=s.acc_out)
        return [s.acc_out]
    si.si_kv_evict(s.kv, s.T, s.budget, sinks=s.sinks, recent=s.recent, path=s.path, n_path=s.n_path, table_out=s.table_out, len_out=s.lens_out)
    return [s.table_out, s.lens_out]


def work(case):
    B, T, Hkv = case["B"], case["T"], case["Hkv"]
    if case["op"] == "evict":
        rows = case["L"] * Hkv
        read = sum(n + case["n_path"] for n in _lens(case))
        # weights of the candidates, the table in and out
        return {"bytes": float(rows * (4 * read + 8 * B * (case["len"] + T))), "flops": 0.0}
    Hq, D = case["Hq"], case["D"]
    if case["op"] == "append":
        return {"bytes": float(B * T * (2 * Hq + 4 * Hkv) * D * 2 + 4 * B * T * case["axes"] + 8 * B * T * Hkv), "flops": float(3 * B * T * (Hq + Hkv) * D)}
    keys = sum(n + T for n in _lens(case)) * Hkv
    if case["op"] == "attend":
        return {"bytes": float(keys * (4 * D + 4) + 4 * B * T * Hq * D + 4 * B * T * Hq), "flops": float(4 * keys * T * (Hq // Hkv) * D)}
    rows = case["n_rows"] * Hq
    return {"bytes": float(keys * (2 * D + 12) + B * rows * (2 * D + 4)), "flops": float(2 * keys * case["n_rows"] * (Hq // Hkv) * D)}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def exact(case, seed):
    if case["op"] == "evict":
        return None  # whole numbers only
    s = prepare(case, seed)
    if s.op == "append":
        return _exact_append(s)
    return _exact_rows(s)


def _exact_append(s):
    B, T, Hq, D = s.q.shape
    half = D // 2
    turn = torch.empty(B, T, half, dtype=torch.complex128, device="cuda")
    pair = 0
    for axis, n in enumerate(s.sections):
        for _ in range(n):
            angle = s.pos[:, :, axis].double() * ROPE_BASE ** (-2.0 * pair / D)
            turn[:, :, pair] = torch.polar(torch.ones_like(angle), angle)
            pair += 1

    def turned(x):
        x = x.double()
        z = torch.complex(x[..., ::2].contiguous(), x[..., 1::2].contiguous()) if s.interleaved else torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
        z = z * turn[:, :, None]
        return torch.view_as_real(z).flatten(-2) if s.interleaved else torch.cat([z.real, z.imag], -1)

    K, V, acc = s.K.double(), s.V.double(), s.acc.double()
    k = turned(s.k)
    for b in range(B):
        n = int(s.lens[0, b])
        for h in range(K.shape[2]):
            slots = s.table[0, b, h, n:n + T].long()
            K[0, b, h, slots] = k[b, :, h]
            V[0, b, h, slots] = s.v[b, :, h].double()
            acc[0, b, h, slots] = 0.0
    return [turned(s.q), K, V, acc]


def _exact_rows(s):
    B, T, Hq, D = s.q.shape
    Hkv = s.K.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    total = s.acc_out.double() if s.op == "weigh" else None
    words = s.mask.cpu().numpy().view(np.uint64)
    for b in range(B):
        n = int(s.lens[0, b])
        sees = torch.zeros(T, n + T, dtype=torch.bool)
        for t in range(T):
            word = int(words[b, t])
            if word:
                sees[t, :n] = True
                sees[t, n:] = torch.tensor([word >> j & 1 for j in range(T)], dtype=torch.bool)
        sees = sees.cuda()
        live = sees.any(1)
        for h in range(Hkv):
            slots = s.table[0, b, h, :n + T].long()
            k = s.K[0, b, h, slots].double()
            q = s.q[b, :, h * G:(h + 1) * G].double()
            z = torch.einsum("tgd,jd->tgj", q, k) * s.scale
            if s.op == "weigh":
                counted = torch.tensor([int(s.rows[b]) >> t & 1 for t in range(T)], dtype=torch.bool, device="cuda")
                p = torch.exp(z - s.lse[b, :, h * G:(h + 1) * G].double()[..., None])
                p = torch.where((sees & counted[:, None])[:, None], p, torch.zeros_like(p))
                total[0, b, h, slots] = s.acc[0, b, h, slots].double() + p.sum((0, 1))
                continue
            z = torch.where(sees[:, None], z, torch.full_like(z, -math.inf))[live]
            lse[b, live, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[b, live, h * G:(h + 1) * G] = torch.softmax(z, -1) @ s.V[0, b, h, slots].double()
    return [total] if s.op == "weigh" else [out, lse]
