"""Decoding with drafted trees over an evicting key/value cache, next to the sparse FFN.

A small decoder with random weights: per layer attention over the cache
(si_kv_append, si_tree_attention, si_kv_accumulate) and a SelectInfer FFN on a
computed set (si_sparse_ffn_decode); once a step si_kv_evict takes the
accepted path into the cache and keeps it within a budget. A step runs the
pending token and a tree of guesses for what follows it; the guesses that the
model itself would have taken are accepted.

    python examples/draft_decode.py [--steps 64] [--budget 96] [--plain]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import activation_sparse_gb300 as si

# The tree of a step: node 0 is the pending token, then three guesses and one more behind each.
PARENTS = [-1, 0, 0, 0, 1, 2, 3]


class Model:
    """Random weights, and what a program keeps: packed FFN layers, computed sets, the cache, rotary positions."""

    def __init__(self, seed=0, layers=2, d=256, neurons=1024, heads=4, kv_heads=2, head_dim=64, vocab=24, slots=512):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = torch.bfloat16
        rnd = lambda *shape, scale: (torch.randn(*shape, generator=g, device="cuda") * scale).to(bf)  # noqa: E731
        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab
        self.emb, self.head = rnd(vocab, d, scale=1.0), rnd(vocab, d, scale=1.0).float()
        self.qkv = [rnd(d, (heads + 2 * kv_heads) * head_dim, scale=d ** -0.5) for _ in range(layers)]
        self.out = [rnd(heads * head_dim, d, scale=4 * (heads * head_dim) ** -0.5) for _ in range(layers)]
        self.ffn, self.S = [], []
        for _ in range(layers):
            Wg, Wu, Wd = rnd(neurons, d, scale=d ** -0.5), rnd(neurons, d, scale=d ** -0.5), rnd(d, neurons, scale=neurons ** -0.5)
            score = torch.rand(neurons, generator=g, device="cuda")
            layer = si.si_pack_loaded(Wg, Wu, Wd, score, score, 0.7, 0.4)
            self.ffn.append(layer)
            self.S.append(torch.arange(0, layer.n_loaded, 2, dtype=torch.int32, device="cuda"))  # the computed set
        self.K = torch.zeros(layers, 1, kv_heads, slots, head_dim, dtype=bf, device="cuda")
        self.V = torch.zeros_like(self.K)
        table = torch.arange(slots, dtype=torch.int32, device="cuda").expand(layers, 1, kv_heads, slots).contiguous()
        acc = torch.zeros(layers, 1, kv_heads, slots, device="cuda")
        self.cache = si.si_kv_create(self.K, self.V, table, torch.zeros(layers, 1, dtype=torch.int32, device="cuda"), acc)
        self.rope = si.si_rope_create(head_dim, base=10000.0)

    def _ffn(self, i, x):
        T, n = x.shape[0], self.S[i].numel()
        S = self.S[i].repeat(T, 1)
        if T > 1:
            si.si_decode_plan(self.ffn[i], S, n, T)
        return si.si_sparse_ffn_decode(self.ffn[i], S, n, T, x, torch.empty(T, x.shape[1], device="cuda"))

    def forward(self, tokens, position, words):
        """Logits [T][vocab] of the new nodes; leaves their keys in the cache's first free slots. Also what
        si_kv_accumulate needs once it is known which nodes count."""
        T, H, Hk, D = tokens.numel(), self.heads, self.kv_heads, self.head_dim
        pos = position.to(torch.int32).view(1, T, 1)
        h = self.emb[tokens].float()
        seen = []
        for i in range(len(self.ffn)):
            x = torch.nn.functional.rms_norm(h, (h.shape[1],)).to(torch.bfloat16)
            qkv = (x @ self.qkv[i]).view(1, T, H + 2 * Hk, D)
            q = torch.empty(1, T, H, D, dtype=torch.bfloat16, device="cuda")
            si.si_kv_append(self.cache, self.rope, qkv[:, :, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:], pos, q, layer=i)
            o, lse = torch.empty_like(q), torch.empty(1, T, H, device="cuda")
            si.si_tree_attention(self.cache, q, o, mask=words, lse=lse, layer=i)
            seen.append((q, lse))
            h = h + (o.view(T, H * D) @ self.out[i]).float()
            h = h + self._ffn(i, torch.nn.functional.rms_norm(h, (h.shape[1],)).to(torch.bfloat16))
        return torch.nn.functional.rms_norm(h, (h.shape[1],)) @ self.head.T, seen

    def keep(self, T, path, words, seen, budget, sinks=4, recent=32):
        """The nodes of `path` stay: their attention counts, and the cache is brought within the budget."""
        rows = torch.tensor([sum(1 << n for n in path)], dtype=torch.int64, device="cuda")
        if budget:
            for i, (q, lse) in enumerate(seen):
                si.si_kv_accumulate(self.cache, q, lse, mask=words, rows=rows, layer=i)
        listed = torch.tensor([path + [0] * (T - len(path))], dtype=torch.int32, device="cuda")
        count = torch.tensor([len(path)], dtype=torch.int32, device="cuda")
        si.si_kv_evict(self.cache, T, budget, sinks=sinks, recent=recent, path=listed, n_path=count)


def words_of(parents):
    """Ancestor words int64 [1][T]: bit j of word t says that node t sees node j."""
    words = []
    for t, p in enumerate(parents):
        words.append(1 << t | (words[p] if p >= 0 else 0))
    return torch.tensor([words], dtype=torch.int64, device="cuda")


def decode(model, prompt, steps, budget=0, draft=True, seed=1):
    """`steps` tokens after the prompt, greedily, and how many were accepted a step on average."""
    guess = torch.Generator().manual_seed(seed)
    chain = lambda T: torch.arange(T, device="cuda")  # noqa: E731
    done = 0
    for at in range(0, len(prompt), 8):
        part = torch.tensor(prompt[at:at + 8], device="cuda")
        words = torch.tensor([[(2 << t) - 1 for t in range(part.numel())]], dtype=torch.int64, device="cuda")
        logits, seen = model.forward(part, done + chain(part.numel()), words)
        model.keep(part.numel(), list(range(part.numel())), words, seen, budget)
        done += part.numel()
    pending, got, runs = int(logits[-1].argmax()), [], 0
    parents = PARENTS if draft else [-1]
    words = words_of(parents)
    depth = torch.tensor([bin(int(w)).count("1") - 1 for w in words[0].tolist()], device="cuda")
    while len(got) < steps:
        guesses = torch.randperm(model.vocab, generator=guess)[:len(parents) - 1].tolist()
        tokens = [pending] + guesses
        logits, seen = model.forward(torch.tensor(tokens, device="cuda"), done + depth, words)
        wanted = logits.argmax(-1).tolist()
        path = [0]
        while True:  # a guess stands if it is what the model wants after the node before it
            follow = [t for t, p in enumerate(parents) if p == path[-1] and tokens[t] == wanted[path[-1]]]
            if not follow:
                break
            path.append(follow[0])
        model.keep(len(parents), path, words, seen, budget)
        got += [tokens[t] for t in path]
        done, pending, runs = done + len(path), wanted[path[-1]], runs + 1
    return got[:steps], len(got) / runs


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--budget", type=int, default=96)
    ap.add_argument("--plain", action="store_true", help="one token a step")
    a = ap.parse_args()
    model = Model()
    tokens, a_step = decode(model, [t * 7 % 24 for t in range(40)], a.steps, a.budget, not a.plain)
    print("tokens", tokens)
    print("%.2f tokens a step, %d keys a list, device error word %#x"
          % (a_step, int(model.cache.lens[0, 0]), si.si_device_error()))


if __name__ == "__main__":
    main()
