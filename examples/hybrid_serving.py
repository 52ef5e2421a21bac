"""A Gated Delta Net layer and a softmax-attention layer served end to end: prompts, draft trees, single tokens.

    python examples/hybrid_serving.py

Two layers with random weights take two prompts, verify a draft tree each (the accepted tokens are a path through
tokens that are rejected), commit the accepted paths, and go on by single tokens.  The first layer keeps a state
(``gdn_prefill``, ``gdn_tree_verify``, ``gdn_tree_commit``, ``gdn_decode``), the second a paged key-value cache
(``gdn_kv_append``, ``gdn_kv_attend``, ``gdn_kv_commit``, ``gdn_kv_decode``); both take the same requests, tree
descriptors and paths.  The same tokens as one prompt give the same outputs; the largest difference is printed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.layer_serving import Layer  # noqa: E402
from gated_delta_net_gb300 import binding as gb  # noqa: E402


class Attention:
    """Weights, cache and forward passes of one attention layer (bf16)."""

    def __init__(self, width=512, n_q_heads=8, n_kv_heads=2, d=64, rot=32, page=16, requests=2, pages=8, positions=128, seed=7):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (scale * torch.randn(*shape, device="cuda", generator=gen)).to(torch.bfloat16)

        self.hq, self.hkv, self.d = n_q_heads, n_kv_heads, d
        self.qkv = normal(width, (n_q_heads + 2 * n_kv_heads) * d, scale=width ** -0.5)
        self.out = normal(n_q_heads * d, width, scale=(n_q_heads * d) ** -0.5)
        self.q_norm, self.k_norm = (1.0 + 0.1 * normal(d, scale=1.0)).to(torch.bfloat16), (1.0 + 0.1 * normal(d)).to(torch.bfloat16)
        self.next_norm = torch.ones(width, device="cuda")
        # far positions' angles in 64 bits
        angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float().cuda()
        self.k = torch.empty(requests * pages, page, n_kv_heads, d, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        self.table = torch.randperm(requests * pages, device="cuda", generator=gen).to(torch.int32).view(requests, pages).contiguous()
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")

    @property
    def cache(self):
        return self.k, self.v, self.table, self.lens

    def append(self, n, offsets, depth, status):
        """New tokens into the cache; the queries."""
        T, rows = n.shape[0], n @ self.qkv
        q, k, v = (rows[:, a * self.d:b * self.d].view(T, b - a, self.d)
                   for a, b in ((0, self.hq), (self.hq, self.hq + self.hkv), (self.hq + self.hkv, self.hq + 2 * self.hkv)))
        return gb.gdn_kv_append(q, k, v, *self.cache, token_offsets=offsets, depth=depth, cos_sin=self.cos_sin, q_weight=self.q_norm,
                                k_weight=self.k_norm, dev_status=status)

    def after(self, x, o):
        return gb.gdn_residual_norm(x, o.view(x.shape[0], -1) @ self.out, self.next_norm, scale=0.5)

    def several(self, x, n, offsets, longest, status, mask=None, depth=None):
        """Prompts (no mask), or draft trees."""
        q = self.append(n, offsets, depth, status)
        return self.after(x, gb.gdn_kv_attend(q, *self.cache, offsets, longest, anc_mask=mask, scale=self.d ** -0.5, dev_status=status))

    def tokens(self, x, n, status):
        q = self.append(n, None, None, status)
        return self.after(x, gb.gdn_kv_decode(q, *self.cache, scale=self.d ** -0.5, dev_status=status))


def run(prompt_lengths=(50, 20), paths=((0, 2, 3, 6), (1, 2)), nodes=(8, 5), singles=4, seed=0):
    """The largest difference, relative to the largest value, between serving in steps and in one prompt."""
    B, status = len(prompt_lengths), gb.new_status()
    gdn, attention, at_once = Layer(seed=seed), Attention(), Attention()
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    lengths = [p + len(a) + singles for p, a in zip(prompt_lengths, paths)]
    xs = [torch.randn(n, gdn.width, device="cuda", generator=gen).to(torch.bfloat16) for n in lengths]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    offsets = lambda ns: ints([sum(ns[:i]) for i in range(len(ns) + 1)])  # noqa: E731
    normed = lambda x: gb.gdn_residual_norm(x, torch.zeros_like(x), gdn.next_norm)[1]  # noqa: E731
    states = lambda: torch.full((B, gdn.hv, gdn.d, gdn.d), float("nan"), device="cuda")  # noqa: E731
    slots, fresh = ints(range(B)), ints([1] * B)

    def prompts(layer, S, parts, counts):
        x = torch.cat(parts)
        h, n = gdn.prompts(x, normed(x), offsets(counts), max(counts), S, slots, fresh, status)
        h, _ = layer.several(h, n, offsets(counts), max(counts), status)
        layer.lens += ints(counts)
        return h.split(counts)

    whole = prompts(at_once, states(), xs, lengths)

    S = states()
    got = [prompts(attention, S, [x[:p] for x, p in zip(xs, prompt_lengths)], list(prompt_lengths))]
    # the drafts: the accepted tokens along a path, rejected ones beside it
    parts, parents = [], []
    for b, path in enumerate(paths):
        x = torch.randn(nodes[b], gdn.width, device="cuda", generator=gen).to(torch.bfloat16)
        x[list(path)] = xs[b][prompt_lengths[b]:prompt_lengths[b] + len(path)]
        parts.append(x)
        before = dict(zip(path[1:], path))
        parents += [before.get(i, -1 if i == path[0] or i == 0 else i - 1) for i in range(nodes[b])]
    x, node_offsets, parent = torch.cat(parts), offsets(nodes), ints(parents)
    path_offsets, path = offsets([len(p) for p in paths]), ints([i for p in paths for i in p])
    mask, depth = gb.gdn_tree_build_desc(parent, node_offsets, max(nodes), dev_status=status)
    h, n = gdn.draft(x, normed(x), node_offsets, parent, path_offsets, path, max(nodes), S, status)
    h, _ = attention.several(h, n, node_offsets, max(nodes), status, mask=mask, depth=depth)
    attention.lens = gb.gdn_kv_commit(*attention.cache, node_offsets, path_offsets, path, dev_status=status)
    got.append([h.split(list(nodes))[b][list(p)] for b, p in enumerate(paths)])
    for t in range(singles):
        x = torch.stack([a[p + len(q) + t] for a, p, q in zip(xs, prompt_lengths, paths)])
        h, n = gdn.tokens(x, normed(x), S, slots, status)
        h, _ = attention.tokens(h, n, status)
        attention.lens += 1
        got.append(h.split(1))
    gb.check_status(status)
    steps, once = (torch.cat([torch.cat([g[b] for g in part]) for b in range(B)]).float() for part in (got, [whole]))
    return float((steps - once).abs().max() / once.abs().max())


if __name__ == "__main__":
    print("%.2e off one prompt's" % run())
