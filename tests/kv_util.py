"""Plain 64-bit definitions of the key/value cache operators, in numpy, and
the inputs of their tests. Shares no code with the library."""
import math

import numpy as np

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}  # half a step, relative


def trees(rng, B, T, nodes=None):
    """Ancestor words uint64 [B][T] of random trees; nodes[b] real nodes, the rest padding (0)."""
    words = np.zeros((B, T), np.uint64)
    for b in range(B):
        for t in range(T if nodes is None else nodes[b]):
            parent = rng.integers(-1, t) if t else -1
            words[b, t] = np.uint64(1 << t) | (words[b, parent] if parent >= 0 else np.uint64(0))
    return words


def chain(B, T):
    return np.array([[(2 << t) - 1 for t in range(T)]] * B, dtype=np.uint64)


def tables(rng, lead, cap, n_slots):
    """Distinct random slots for every list."""
    out = np.empty(lead + (cap,), np.int32)
    for i in np.ndindex(*lead):
        out[i] = rng.permutation(n_slots)[:cap]
    return out


def angles(pos, inv_freq, axis):
    """cos, sin [..., pairs] of pos [..., axes]. The products are reduced modulo one turn in
    128-bit integers, so that far positions lose nothing."""
    pos = np.asarray(pos, np.int64)
    two_pi = 8 * sum((-1) ** k * (4 * _atan_inv(5) if k == 0 else _atan_inv(239)) for k in (0, 1))  # 2 pi, 2^-160 steps
    turn = []
    for f in inv_freq:
        num, den = float(f).as_integer_ratio()
        turn.append((num << 320) // (den * two_pi) % (1 << 160))  # fraction of a turn, 2^-160 steps
    ang = np.empty(pos.shape[:-1] + (len(turn),))
    for i, (t, a) in enumerate(zip(turn, axis)):
        flat = [(int(p) * t) % (1 << 160) for p in pos[..., a].reshape(-1)]
        ang[..., i] = (np.array([float(x - (1 << 160) if x >> 159 else x) for x in flat]) * 2.0 ** -160).reshape(pos.shape[:-1])
    return np.cos(2 * math.pi * ang), np.sin(2 * math.pi * ang)


def _atan_inv(x, bits=160):
    """atan(1/x) in steps of 2^-bits (Gregory's series in integers; Machin: pi/4 = 4 atan(1/5) - atan(1/239))."""
    t = (1 << (bits + 16)) // x
    total, k, sign = 0, 1, 1
    while t:
        total += sign * (t // k)
        t //= x * x
        k += 2
        sign = -sign
    return total >> 16


def rotate(x, cos, sin, interleaved):
    """x [B, T, H, D] float64; cos, sin [B, T, pairs]."""
    n = cos.shape[-1]
    y = x.copy()
    c, s = cos[:, :, None], sin[:, :, None]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * c - b * s, b * c + a * s
    return y


def sees(word, n, T):
    """Which of the n + T entries a node with this ancestor word sees."""
    if int(word) == 0:
        return np.zeros(n + T, bool)
    return np.concatenate([np.ones(n, bool), np.array([int(word) >> j & 1 for j in range(T)], bool)])


def attend(q, K, V, table, lens, words, scale):
    """out, lse, and per output the sum of weight * |v| (for error bounds), float64."""
    B, T, Hq, D = q.shape
    G = Hq // K.shape[1]
    out, mag = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D))
    lse = np.full((B, T, Hq), -np.inf)
    for b in range(B):
        n = int(lens[b])
        for h in range(K.shape[1]):
            slots = np.arange(n + T) if table is None else table[b, h, :n + T]
            for t in range(T):
                vis = sees(words[b, t], n, T)
                if not vis.any():
                    continue
                k, v = K[b, h, slots[vis]], V[b, h, slots[vis]]
                for g in range(G):
                    z = scale * (k @ q[b, t, h * G + g])
                    top = z.max()
                    e = np.exp(z - top)
                    lse[b, t, h * G + g] = top + np.log(e.sum())
                    p = e / e.sum()
                    out[b, t, h * G + g] = p @ v
                    mag[b, t, h * G + g] = p @ np.abs(v)
    return out, lse, mag


def weigh(q, K, table, lens, words, rows, lse, acc, scale):
    """acc with the counted rows' weights added, float64 (all slots)."""
    B, T, Hq, D = q.shape
    G = Hq // K.shape[1]
    got = acc.astype(np.float64).copy()
    for b in range(B):
        n = int(lens[b])
        for h in range(K.shape[1]):
            slots = np.arange(n + T) if table is None else table[b, h, :n + T]
            for t in range(T):
                vis = sees(words[b, t], n, T)
                if not vis.any() or not (rows is None or int(rows[b]) >> t & 1):
                    continue
                for g in range(G):
                    if lse[b, t, h * G + g] == -np.inf:
                        continue
                    z = scale * (K[b, h, slots[vis]] @ q[b, t, h * G + g])
                    got[b, h, slots[vis]] += np.exp(z - lse[b, t, h * G + g])
    return got


def evict(table, lens, acc, T, path, n_path, budget, sinks, recent):
    """New table and lens, by sorting."""
    table, lens_out = table.copy(), lens.copy()
    L, B, H, cap = table.shape
    for l in range(L):
        for b in range(B):
            n = int(lens[l, b])
            np_ = T if n_path is None else int(n_path[b])
            nodes = list(range(np_)) if path is None else [int(x) for x in path[b, :np_]]
            for h in range(H):
                old = table[l, b, h].copy()
                cand = list(old[:n]) + [old[n + x] for x in nodes]
                rest = [old[n + x] for x in range(T) if x not in nodes]
                kept = list(range(len(cand)))
                if budget > 0 and len(cand) > budget:
                    m = len(cand)
                    safe = [c for c in range(m) if c < sinks or c >= m - recent]
                    weight = {c: acc[l, b, h, cand[c]] for c in range(m)}
                    weight = {c: -np.inf if np.isnan(w) else w for c, w in weight.items()}
                    nan = {c: bool(np.isnan(acc[l, b, h, cand[c]])) for c in range(m)}
                    others = sorted((c for c in range(m) if c not in set(safe)), key=lambda c: (nan[c], -weight[c], c))
                    kept = sorted(safe + others[:budget - len(safe)])
                keep = set(kept)
                gone = [c for c in range(len(cand)) if c not in keep]
                table[l, b, h, :n + T] = [cand[c] for c in kept] + [cand[c] for c in gone] + rest
                lens_out[l, b] = len(kept)
    return table, lens_out
