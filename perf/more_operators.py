"""Cases of the operators over a key/value cache in 8 bits, and of the log probabilities that decide on drafted tokens.

An 8-bit cache holds keys and values as e4m3 codes with a power-of-two scale (a biased exponent byte, E8M0) for each
block of slots of a head: code * 2^(byte - 127) is what the cache stands for. With blocks of one slot `si_kv_append`
chooses the scale from the row that it writes; with larger blocks the scales are the program's, calibrated beforehand.
`si_tree_attention` and `si_kv_accumulate` read such a cache as they read one in 16 bits. `si_token_logprobs` takes a
step's logits: the log probabilities of the drafted tokens, the entropy, and each node's best alternatives.

Each case names its operator in "op". Where `own` is false, `run` computes it with elementary torch operations;
where it is true, it calls the framework.
"""
import math
import types

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 number
# exponents of a scale: every code stands for a number of the cache's type
EXPONENTS = {"bf16": (-124, 119), "fp16": (-15, 7)}
ROPE_BASE = 500000.0


def listed():
    return [
        # one new token of one sequence: the smallest append, all latency
        dict(name="append-token", op="append", B=1, T=1, Hq=32, Hkv=8, D=64, axes=1, interleaved=False, dtype="bf16", far=4096, block=1),
        # drafted trees of a batch, calibrated scales, one a head
        dict(name="append-tree", op="append", B=8, T=33, Hq=32, Hkv=8, D=128, axes=1, interleaved=True, dtype="fp16", far=1000000, block=65536),
        # a prompt with images: three axes
        dict(name="append-prompt", op="append", B=1, T=8192, Hq=32, Hkv=8, D=128, axes=3, interleaved=False, dtype="bf16", far=16384, block=1),
        # one token over a short chat, an evicted cache
        dict(name="attend-token", op="attend", B=1, T=1, Hq=32, Hkv=8, D=64, len=1000, ragged=False, order="evicted", dtype="bf16", block=1),
        # decoding for a batch of unequal contexts
        dict(name="attend-batch", op="attend", B=16, T=1, Hq=32, Hkv=8, D=128, len=4097, ragged=True, order="evicted", dtype="fp16", block=16),
        # wide trees of a batch: the most rows a key meets
        dict(name="attend-wide", op="attend", B=8, T=64, Hq=32, Hkv=8, D=128, len=8192, ragged=True, order="evicted", dtype="fp16", block=1 << 20),
        # one token over a long document that never evicted
        dict(name="attend-long", op="attend", B=1, T=1, Hq=32, Hkv=8, D=128, len=131071, ragged=False, order="fresh", dtype="bf16", block=1),
        # weights of one token's attention
        dict(name="weigh-token", op="weigh", B=1, T=1, n_rows=1, Hq=32, Hkv=8, D=64, len=4095, ragged=False, order="evicted", dtype="bf16", block=1),
        # weights of the accepted tokens of a batch of trees
        dict(name="weigh-tree", op="weigh", B=8, T=16, n_rows=4, Hq=32, Hkv=8, D=128, len=16384, ragged=True, order="evicted", dtype="fp16", block=64),
        # the next token of one sequence, with its best alternatives
        dict(name="logprobs-token", op="logprobs", N=1, V=32768, M=1, K=8, dtype="fp32", masked=False),
        # the nodes of a batch of drafted trees: their children's tokens, a constrained vocabulary of odd size
        dict(name="logprobs-tree", op="logprobs", N=128, V=50001, M=4, K=4, dtype="bf16", masked=True),
        # scoring a prompt: every position's own token
        dict(name="logprobs-prompt", op="logprobs", N=2048, V=131072, M=1, K=1, dtype="bf16", masked=False),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of its range."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weigh", "logprobs"])
    if op == "logprobs":
        V = _log(rng, 100, 200000)
        return dict(op=op, N=_log(rng, 1, min(4096, 2 ** 28 // V)), V=V, M=rng.choice([0, 1, 1, 3, 8]), K=min(V, rng.choice([0, 1, 2, 5, 20, 32])),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), masked=rng.choice([False, True]))
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    block = rng.choice([1, 1, 1, 16, 128, 1 << 20])
    if op == "append":
        B = rng.choice([1, 2, 3, 8])
        T = _log(rng, 1, 8192 // B)
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=min(D, 128), axes=rng.choice([1, 2, 3]), interleaved=rng.choice([False, True]),
                    dtype=dtype, far=_log(rng, 100, 2000000), block=block)
    B = rng.choice([1, 1, 2, 4, 7, 16])
    T = rng.choice([1, 1, 1, 2, 5, 8, 16, 31, 64])
    top = min(131072, 2 ** 27 // (B * Hkv * D), 2 ** 33 // (B * Hkv * G * T * D))  # at most the long document's keys
    n = _log(rng, 1, top)
    case = dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, len=n, ragged=rng.choice([False, True]), order=rng.choice(["evicted", "fresh"]),
                dtype=dtype, block=block)
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


def _blocks(n_slots, block):
    return (n_slots + block - 1) // block


def _pool(gen, B, Hkv, n_slots, D, block, dtype):
    """Codes [1, B, Hkv, n_slots, D] and scale bytes [1, B, Hkv, blocks] of normal keys, each head of a size of its own."""
    size = torch.exp(0.7 * torch.randn(1, B, Hkv, 1, 1, generator=gen, device="cuda"))
    x = size * torch.randn(1, B, Hkv, n_slots, D, generator=gen, device="cuda")
    n = _blocks(n_slots, block)
    at = torch.arange(n_slots, device="cuda") // block
    top = torch.zeros(1, B, Hkv, n, device="cuda").scatter_reduce_(3, at.expand(1, B, Hkv, -1), x.abs().amax(-1), "amax")
    byte = _scale_byte(top, dtype)
    return (x / _power(byte[..., at])[..., None]).to(E4M3), byte


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = types.SimpleNamespace(op=case["op"])
    rnd = lambda *shape, dtype=torch.float32: torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    if s.op == "logprobs":
        N, V, M, K = case["N"], case["V"], case["M"], case["K"]
        # distributions from nearly even to nearly decided
        s.logits = (rnd(N, V) * (1.0 + 3.0 * torch.rand(N, 1, generator=gen, device="cuda"))).to(DTYPES[case["dtype"]])
        if case["masked"]:
            s.logits.masked_fill_(torch.rand(V, generator=gen, device="cuda") < 0.1, -math.inf)
        s.targets = torch.randint(0, V, (N, M), generator=gen, device="cuda", dtype=torch.int32)
        s.targets.masked_fill_(torch.rand(N, M, generator=gen, device="cuda") < 0.1, -1)  # nodes with fewer children
        s.temperature, s.K = 0.8, K
        s.logp, s.entropy = torch.empty(N, M, device="cuda"), torch.empty(N, device="cuda")
        s.top_logp, s.top_ids = torch.empty(N, K, device="cuda"), torch.empty(N, K, dtype=torch.int32, device="cuda")
        return s
    B, T, Hq, Hkv, D, block = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"], case["block"]
    dtype = DTYPES[case["dtype"]]
    s.block, s.limits = block, EXPONENTS[case["dtype"]]
    if s.op == "append":
        entries = T + 64
        s.K, s.V = (torch.zeros(1, B, Hkv, entries, D, device="cuda").to(E4M3) for _ in range(2))
        # calibrated: normal rows reach some five sizes
        n = _blocks(entries, block)
        s.k_scale, s.v_scale = (torch.full((1, B, Hkv, n), 127 - 6, dtype=torch.uint8, device="cuda") for _ in range(2))
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
            s.kv = si.si_kv_create(s.K, s.V, s.table, s.lens, s.acc, k_scale=s.k_scale, v_scale=s.v_scale, block=block, dtype=dtype)
        return s
    cap = case["len"] + T
    s.K, s.k_scale = _pool(gen, B, Hkv, cap, D, block, case["dtype"])
    s.V, s.v_scale = _pool(gen, B, Hkv, cap, D, block, case["dtype"])
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
        s.lse = torch.cat([_softmax(_scores(s.q[b:b + 1], s.K[:, b:b + 1], s.k_scale[:, b:b + 1], s.block, s.table[:, b:b + 1], s.scale),
                                    _visible(s.lens[:, b:b + 1], s.mask[b:b + 1], cap))[1] for b in range(B)])
    if own:
        import activation_sparse_gb300 as si
        s.kv = si.si_kv_create(s.K, s.V, s.table, s.lens, s.acc, k_scale=s.k_scale, v_scale=s.v_scale, block=block, dtype=dtype)
    return s


# ------------------------------------------------------------------ the plain forms

def _scale_byte(top, dtype):
    """The smallest power of two whose 448-fold holds `top`, within the type's limits, as a biased exponent."""
    lo, hi = EXPONENTS[dtype] if isinstance(dtype, str) else dtype
    m, x = torch.frexp(top)  # top = m * 2^x, m in [1/2, 1); 448 = 7/8 * 2^9
    e = torch.where(top == 0, lo, x - 9 + (m > 0.875).int()).clamp(lo, hi) + 127
    return torch.where(top.isfinite(), e, 255).to(torch.uint8)


def _power(byte):
    """What a scale byte stands for: 2^(byte - 127), 255 is NaN."""
    return torch.where(byte == 255, math.nan, (byte.to(torch.int32) << 23).view(torch.float32))


def _rotate(x, cos, sin, interleaved):
    """x [B, T, H, D] with the angles' cos and sin [B, T, 1, D / 2], in 32 bits."""
    f = x.float()
    half = f.shape[-1] // 2
    a, b = (f[..., 0::2], f[..., 1::2]) if interleaved else (f[..., :half], f[..., half:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    return torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)


def _store(s, pool, scale, x, slot):
    """Rows x [B, Hkv, T, D] of 32 bits into their slots: codes, and in blocks of one slot the scale."""
    if s.block == 1:
        byte = _scale_byte(x.abs().amax(-1), s.limits)
        scale[0].scatter_(2, slot, byte)
    else:
        byte = scale[0].gather(2, slot // s.block)
    code = (x / _power(byte)[..., None]).clamp(-TOP, TOP).to(E4M3)
    rows = slot[..., None].expand(-1, -1, -1, x.shape[-1])
    pool[0].view(torch.uint8).scatter_(2, rows, code.view(torch.uint8))


def _append(s):
    angle = s.pos.double()[..., s.axis] * s.inv_freq  # far positions: the angle needs 64 bits
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    T = s.pos.shape[1]
    at = s.lens[0, :, None].long() + torch.arange(T, device="cuda")
    slot = s.table[0].gather(2, at[:, None, :].expand(-1, s.table.shape[2], -1)).long()
    _store(s, s.K, s.k_scale, _rotate(s.k, cos, sin, s.interleaved).transpose(1, 2), slot)
    _store(s, s.V, s.v_scale, s.v.float().transpose(1, 2), slot)
    s.acc[0].scatter_(2, slot, 0.0)
    s.q_out.copy_(_rotate(s.q, cos, sin, s.interleaved))
    return _appended(s)


def _appended(s):
    return [s.q_out, s.K, s.V, s.k_scale.view(torch.float8_e8m0fnu), s.v_scale.view(torch.float8_e8m0fnu), s.acc]


def _visible(lens, words, entries):
    """Which list entries each drafted node sees: bool [B, T, entries]."""
    i = torch.arange(entries, device="cuda")
    j = i[None] - lens[0, :, None].long()  # the draft's own index, negative for a cached key
    T = words.shape[1]
    bit = (words[:, :, None] >> j.clamp(0, T - 1)[:, None, :]) & 1
    return ((j < 0)[:, None, :] | ((j < T)[:, None, :] & (bit != 0))) & (words != 0)[:, :, None]


def _listed(pool, scale, block, table):
    """What the pool's rows stand for, in list order, in 32 bits."""
    slot = table[0].long()
    rows = pool[0].view(torch.uint8).gather(2, slot[..., None].expand(-1, -1, -1, pool.shape[-1])).view(E4M3).float()
    return rows * _power(scale[0].gather(2, slot // block))[..., None]


def _scores(q, K, k_scale, block, table, scale):
    """Scaled products [B, Hkv, T, G, entries]."""
    B, T, Hq, D = q.shape
    Hkv = K.shape[2]
    rows = q.float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    return ((rows @ _listed(K, k_scale, block, table).transpose(2, 3)) * scale).view(B, Hkv, T, Hq // Hkv, -1)


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
    (p, total), lse = _softmax(_scores(s.q, s.K, s.k_scale, s.block, s.table, s.scale), _visible(s.lens, s.mask, s.table.shape[-1]))
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = p.flatten(2, 3) @ _listed(s.V, s.v_scale, s.block, s.table)
    s.out.copy_(o.view(B, -1, T, Hq // s.K.shape[2], D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D))
    s.lse.copy_(lse)
    return [s.out, s.lse]


def _weigh(s):
    T = s.q.shape[1]
    entries = s.table.shape[-1]
    scores = _scores(s.q, s.K, s.k_scale, s.block, s.table, s.scale)
    B = s.q.shape[0]
    visible = _visible(s.lens, s.mask, entries) & ((s.rows[:, None] >> torch.arange(T, device="cuda")) & 1 != 0)[:, :, None]
    lse = s.lse.view(B, T, -1, scores.shape[3]).permute(0, 2, 1, 3)[..., None]
    w = (scores - lse).exp_().masked_fill_(~visible[:, None, :, None], 0.0).sum((2, 3))
    slot = s.table[0].long()
    listed_now = torch.arange(entries, device="cuda") < s.lens[0, :, None, None] + T
    s.acc_out[0].scatter_(2, slot, torch.where(listed_now, s.acc[0].gather(2, slot) + w, s.acc_out[0].gather(2, slot)))
    return [s.acc_out]


def _logprobs(s):
    z = s.logits.float() / s.temperature
    top = z.amax(-1, keepdim=True)
    shifted = z - top
    p = shifted.exp()
    total = p.sum(-1, keepdim=True)
    rest = total.log()
    # an entry without probability adds nothing: 0 * -inf is left out
    s.entropy.copy_((rest - torch.where(p > 0, p * shifted, 0.0).sum(-1, keepdim=True) / total)[:, 0])
    logp = shifted - rest
    t = s.targets.long()
    s.logp.copy_(torch.where(t < 0, -math.inf, logp.gather(1, t.clamp(min=0))))
    # whole numbers in the order of the logits, ties to the lower id
    bits = (s.logits.float() + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32 - torch.arange(z.shape[1], device="cuda")
    ids = order.topk(s.K, -1).indices
    s.top_ids.copy_(ids)
    s.top_logp.copy_(logp.gather(1, ids))
    return [s.logp, s.entropy, s.top_logp, s.top_ids]


def run(state):
    s = state
    if not own:
        return {"append": _append, "attend": _attend, "weigh": _weigh, "logprobs": _logprobs}[s.op](s)
    import activation_sparse_gb300 as si
    if s.op == "append":
        si.si_kv_append(s.kv, s.rope, s.q, s.k, s.v, s.pos, s.q_out)
        return _appended(s)
    if s.op == "attend":
        si.si_tree_attention(s.kv, s.q, s.out, mask=s.mask, lse=s.lse, scale=s.scale)
        return [s.out, s.lse]
    if s.op == "weigh":
        si.si_kv_accumulate(s.kv, s.q, s.lse, mask=s.mask, rows=s.rows, scale=s.scale, acc_out=s.acc_out)
        return [s.acc_out]
    si.si_token_logprobs(s.logits, targets=s.targets, logp=s.logp, entropy=s.entropy, top_logp=s.top_logp, top_ids=s.top_ids,
                         temperature=s.temperature)
    return [s.logp, s.entropy, s.top_logp, s.top_ids]


def work(case):
    if case["op"] == "logprobs":
        N, V, M, K = case["N"], case["V"], case["M"], case["K"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": float(N * (V * size + 8 * M + 4 + 8 * K)), "flops": float(4 * N * V)}
    B, T, Hkv, Hq, D, block = case["B"], case["T"], case["Hkv"], case["Hq"], case["D"], case["block"]
    if case["op"] == "append":
        scales = 2 * B * Hkv * (T if block == 1 else 1)
        return {"bytes": float(B * T * (2 * (2 * Hq + 2 * Hkv) * D + 2 * Hkv * D) + 4 * B * T * case["axes"] + 8 * B * T * Hkv + scales),
                "flops": float(3 * B * T * (Hq + Hkv) * D)}
    listed_now = sum(n + T for n in _lens(case))
    keys, scales = listed_now * Hkv, sum(_blocks(n + T, block) for n in _lens(case)) * Hkv
    if case["op"] == "attend":
        return {"bytes": float(keys * (2 * D + 4) + 2 * scales + 4 * B * T * Hq * D + 4 * B * T * Hq), "flops": float(4 * keys * T * (Hq // Hkv) * D)}
    rows = case["n_rows"] * Hq
    return {"bytes": float(keys * (D + 12) + scales + B * rows * (2 * D + 4)), "flops": float(2 * keys * case["n_rows"] * (Hq // Hkv) * D)}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if s.op == "logprobs":
        return _exact_logprobs(s)
    if s.op == "append":
        return _exact_append(s)
    return _exact_rows(s)


def _exact_logprobs(s):
    N, V = s.logits.shape
    logp, entropy, best = [], [], []
    for at in range(0, N, 64):
        z = s.logits[at:at + 64].double() / s.temperature
        l = z - torch.logsumexp(z, -1, keepdim=True)
        entropy.append(-torch.special.xlogy(l.exp(), l.exp()).sum(-1))
        t = s.targets[at:at + 64]
        logp.append(torch.stack([torch.where(t[:, m] < 0, -math.inf, l[torch.arange(len(l)), t[:, m].long().clamp(min=0)]) for m in range(t.shape[1])], 1)
                    if t.shape[1] else l[:, :0])
        best.append(l.topk(s.K, -1).values)
    return [torch.cat(logp), torch.cat(entropy), torch.cat(best), None]


def _turned(s, x):
    """The rotation as a product of complex numbers."""
    B, T = s.pos.shape[:2]
    D = x.shape[-1]
    half = D // 2
    turn = torch.empty(B, T, half, dtype=torch.complex128, device="cuda")
    pair = 0
    for axis, n in enumerate(s.sections):
        for _ in range(n):
            angle = s.pos[:, :, axis].double() * ROPE_BASE ** (-2.0 * pair / D)
            turn[:, :, pair] = torch.polar(torch.ones_like(angle), angle)
            pair += 1
    x = x.double()
    z = torch.complex(x[..., ::2].contiguous(), x[..., 1::2].contiguous()) if s.interleaved else torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
    z = z * turn[:, :, None]
    return torch.view_as_real(z).flatten(-2) if s.interleaved else torch.cat([z.real, z.imag], -1)


def _exact_append(s):
    """The codes before their rounding: the row over its scale."""
    B, T = s.pos.shape[:2]
    pools = []
    for pool, scale, rows in ((s.K, s.k_scale, _turned(s, s.k)), (s.V, s.v_scale, s.v.double())):
        pool, power = pool.float().double(), torch.exp2(scale.double() - 127)
        for b in range(B):
            n = int(s.lens[0, b])
            for h in range(pool.shape[2]):
                slots = s.table[0, b, h, n:n + T].long()
                row = rows[b, :, h]
                if s.block == 1:
                    lo, hi = s.limits
                    e = torch.ceil(torch.log2(row.abs().amax(-1) / TOP)).clamp(lo, hi)
                    power[0, b, h, slots] = torch.exp2(e)
                pool[0, b, h, slots] = (row / power[0, b, h, slots // s.block][:, None]).clamp(-TOP, TOP)
        pools.append((pool, power))
    acc = s.acc.double()
    for b in range(B):
        n = int(s.lens[0, b])
        acc[0, b].scatter_(1, s.table[0, b, :, n:n + T].long(), 0.0)
    (K, k_power), (V, v_power) = pools
    return [_turned(s, s.q), K, V, k_power, v_power, acc]


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

            def rows(pool, scale):
                power = torch.pow(2.0, scale[0, b, h, torch.div(slots, s.block, rounding_mode="floor")].double() - 127.0)
                return pool[0, b, h].float()[slots].double() * power[:, None]

            k = rows(s.K, s.k_scale)
            q = s.q[b, :, h * G:(h + 1) * G].double()
            z = torch.einsum("tgd,jd->tgj", q, k) * s.scale
            if s.op == "weigh":
                counted = sees & torch.tensor([int(s.rows[b]) >> t & 1 for t in range(T)], dtype=torch.bool, device="cuda")[:, None]
                w = torch.exp(z - s.lse[b, :, h * G:(h + 1) * G].double()[..., None])
                w = torch.where(counted[:, None], w, 0.0).sum((0, 1))
                total[0, b, h, slots] = s.acc[0, b, h, slots].double() + w
                continue
            z = z.masked_fill(~sees[:, None], -math.inf)
            l = torch.logsumexp(z, -1)
            p = torch.exp(z - torch.where(live[:, None], l, 0.0)[..., None])
            out[b, :, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", p, rows(s.V, s.v_scale))
            lse[b, :, h * G:(h + 1) * G] = l
    return [total] if s.op == "weigh" else [out, lse]
