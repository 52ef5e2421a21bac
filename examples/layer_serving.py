"""One Gated Delta Net layer served end to end: prompts, a draft tree, single tokens.

    python examples/layer_serving.py

A layer with random weights takes two prompts through ``gdn_prefill``, verifies and commits a draft (a chain
here, so that the answer is known) with ``gdn_tree_verify`` and ``gdn_tree_commit`` on the states that the
prompts left, and goes on by single tokens with ``gdn_decode``.  ``gdn_qk_gates`` stands before the rule in all
three, ``gdn_norm_gate`` and ``gdn_residual_norm`` after it.  The same tokens as one prompt give the same
outputs; the largest differences are printed.  The projections are plain matrix products of torch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_delta_net_gb300 import binding as gb  # noqa: E402


class Layer:
    """Weights and forward passes of one layer of width ``width`` (bf16)."""

    def __init__(self, width=512, n_k_heads=2, n_v_heads=4, d=128, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (scale * torch.randn(*shape, device="cuda", generator=gen)).to(torch.bfloat16)

        self.hk, self.hv, self.d, self.width = n_k_heads, n_v_heads, d, width
        self.qkvz = normal(width, (2 * n_k_heads + 2 * n_v_heads) * d, scale=width ** -0.5)
        self.ab = normal(width, 2 * n_v_heads, scale=width ** -0.5)
        self.out = normal(n_v_heads * d, width, scale=(n_v_heads * d) ** -0.5)
        self.A_log = torch.zeros(n_v_heads, device="cuda")
        self.dt_bias = torch.full((n_v_heads,), -4.0, device="cuda")
        self.norm, self.next_norm = torch.ones(d, device="cuda"), torch.ones(width, device="cuda")

    def before(self, n):
        """The rule's inputs from normed activations n [T, width]: q, k, g, beta, and v, z as slices of the
        fused projection's rows."""
        T, kw, vw = n.shape[0], self.hk * self.d, self.hv * self.d
        rows, ab = n @ self.qkvz, n @ self.ab
        q, k = rows[:, :kw].view(T, self.hk, self.d), rows[:, kw:2 * kw].view(T, self.hk, self.d)
        v = rows[:, 2 * kw:2 * kw + vw].view(T, self.hv, self.d)
        z = rows[:, 2 * kw + vw:].view(T, self.hv, self.d)
        q, k, g, beta = gb.gdn_qk_gates(q, k, ab[:, :self.hv], ab[:, self.hv:], self.A_log, self.dt_bias)
        return q, k, v, z, g, beta

    def after(self, x, o, z):
        """(residual stream, next layer's normed activations) from the rule's output."""
        y = gb.gdn_norm_gate(o, z, self.norm)
        return gb.gdn_residual_norm(x, y.view(x.shape[0], -1) @ self.out, self.next_norm, scale=0.5)

    def prompts(self, x, n, offsets, longest, S, slots, fresh, status):
        q, k, v, z, g, beta = self.before(n)
        o, _ = gb.gdn_prefill(q, k, v, g, beta, offsets, longest, S0=S, S_new=S, slots=slots, fresh=fresh,
                              scale=self.d ** -0.5, dev_status=status)
        return self.after(x, o, z)

    def tokens(self, x, n, S, slots, status):
        q, k, v, z, g, beta = self.before(n)
        o = gb.gdn_decode(q, k, v, g, beta, S, slots=slots, scale=self.d ** -0.5, dev_status=status)
        return self.after(x, o, z)

    def draft(self, x, n, node_offsets, parent, path_offsets, path, nodes, S, status):
        """Every node's outputs; S [B, Hv, d, d] advances along the accepted paths."""
        q, k, v, z, g, beta = self.before(n)
        v = v.contiguous()
        mask, depth = gb.gdn_tree_build_desc(parent, node_offsets, nodes, dev_status=status)
        o = gb.gdn_tree_verify(q, k, v, g, beta, S, node_offsets, parent, mask, depth, nodes, max_depth=16,
                               scale=self.d ** -0.5, dev_status=status)
        gb.gdn_tree_commit(k, v, g, beta, S, node_offsets, parent, path_offsets, path, nodes, max_path=16, out=S,
                           dev_status=status)
        return self.after(x, o, z)


def run(prompt_lengths=(150, 40), draft=12, singles=5, seed=0):
    """The largest difference, relative to the largest value, between serving in steps and in one prompt:
    (residual stream, final states)."""
    layer = Layer(seed=seed)
    status = gb.new_status()
    B = len(prompt_lengths)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    lengths = [p + draft + singles for p in prompt_lengths]
    xs = [torch.randn(n, layer.width, device="cuda", generator=gen).to(torch.bfloat16) for n in lengths]
    offsets = lambda ns: torch.tensor([0] + list(ns), device="cuda").cumsum(0).to(torch.int32)  # noqa: E731
    cut = lambda a, b: torch.cat([x[p + a:p + b] for x, p in zip(xs, prompt_lengths)])  # noqa: E731
    slots = torch.arange(B, device="cuda", dtype=torch.int32).flip(0).contiguous()
    fresh = torch.ones(B, device="cuda", dtype=torch.int32)

    def normed(x):
        return gb.gdn_residual_norm(x, torch.zeros_like(x), layer.next_norm)[1]

    # all at once
    whole = torch.cat(xs)
    S_whole = torch.full((B, layer.hv, layer.d, layer.d), float("nan"), device="cuda")
    h_whole, _ = layer.prompts(whole, normed(whole), offsets(lengths), max(lengths), S_whole, slots, fresh, status)

    # in steps: prompts, a chain draft that is accepted whole, single tokens
    S = torch.full_like(S_whole, float("nan"))
    x = torch.cat([a[:p] for a, p in zip(xs, prompt_lengths)])
    got = [layer.prompts(x, normed(x), offsets(prompt_lengths), max(prompt_lengths), S, slots, fresh, status)[0].split(list(prompt_lengths))]
    x = cut(0, draft)
    parent = torch.arange(-1, draft - 1, device="cuda", dtype=torch.int32).repeat(B)
    path = torch.arange(draft, device="cuda", dtype=torch.int32).repeat(B)
    nodes = offsets([draft] * B)
    by_request = S[slots.long()].contiguous()
    got.append(layer.draft(x, normed(x), nodes, parent, nodes, path, draft, by_request, status)[0].split([draft] * B))
    S[slots.long()] = by_request
    for t in range(draft, draft + singles):
        x = cut(t, t + 1)
        got.append(layer.tokens(x, normed(x), S, slots, status)[0].split([1] * B))
    gb.check_status(status)
    h = torch.cat([torch.cat([step[b] for step in got]) for b in range(B)])
    far = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())  # noqa: E731
    return far(h, h_whole), far(S, S_whole)


if __name__ == "__main__":
    print("residual stream %.2e, states %.2e off one prompt's" % run())
