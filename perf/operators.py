"""What the layer operators of gated_delta_net_gb300 are measured on: prompts and single tokens through the
gated delta rule, and the norms and gates before and after it.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the end)
or, where `own` is true, calls the framework.  `exact` is the definition in 64 bits.  Head counts and widths are
the ones this repository's workloads use (16 key / 32 value heads of width 128, and the smaller ones it supports);
prompt lengths and hidden widths are generic.
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-6


def listed():
    return [
        # the first request of an idle server: one short prompt, every launch counts
        dict(name="prefill_one_short", op="prefill", lengths="37", hk=16, hv=32, dk=128, dv=128, dtype="bf16", pool=False),
        # one long document: only the heads and the split of its length fill the GPU
        dict(name="prefill_one_long", op="prefill", lengths="16384", hk=16, hv=32, dk=128, dv=128, dtype="bf16", pool=False),
        # a serving step that mixes fresh prompts and continued ones, states in a pool of slots
        dict(name="prefill_ragged_b64", op="prefill", lengths="ragged:64:16:512", hk=16, hv=32, dk=128, dv=128, dtype="bf16",
             pool=True),
        # the 32-bit form, as a numerics check of a model runs it
        dict(name="prefill_f32_b3", op="prefill", lengths="1,300,129", hk=16, hv=16, dk=128, dv=128, dtype="f32", pool=False),
        # one user, one token
        dict(name="decode_b1", op="decode", batch=1, n_states=8, dead=0, hk=16, hv=32, dk=128, dv=128, dtype="bf16"),
        # a full serving batch padded to its graph's size: some rows are not in use
        dict(name="decode_b256", op="decode", batch=256, n_states=300, dead=7, hk=16, hv=32, dk=128, dv=128, dtype="bf16"),
        # norms and gates before the rule: a decode batch, and a prompt's tokens out of one fused projection
        dict(name="qk_gates_t64", op="qk_gates", tokens=64, hk=16, hv=32, dk=128, dv=128, dtype="bf16"),
        dict(name="qk_gates_t16k", op="qk_gates", tokens=16384, hk=16, hv=32, dk=128, dv=128, dtype="bf16"),
        # the gated norm after the rule: a decode batch and a prompt
        dict(name="norm_gate_t64", op="norm_gate", tokens=64, hv=32, dv=128, dtype="bf16", act="silu"),
        dict(name="norm_gate_t16k", op="norm_gate", tokens=16384, hv=32, dv=128, dtype="bf16", act="silu"),
        # the residual stream between blocks: a decode batch, and a prompt with a norm on the block's output as well
        dict(name="residual_norm_t64", op="residual_norm", tokens=64, width=4096, dtype="bf16", post=False),
        dict(name="residual_norm_t8k", op="residual_norm", tokens=8192, width=5120, dtype="bf16", post=True),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "qk_gates", "norm_gate", "residual_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 2, 2, 4])
    if op in ("prefill", "decode"):
        dk, dv = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (128, 64), (32, 16)])
        if op == "decode":
            batch = _log_uniform(rng, 1, 200)
            return dict(op=op, batch=batch, n_states=batch + rng.randint(0, 40), dead=rng.randint(0, batch // 8), hk=hk, hv=hv,
                        dk=dk, dv=dv, dtype=dtype)
        most = 12000 if dtype == "bf16" else 3000
        total, n = _log_uniform(rng, 1, most), _log_uniform(rng, 1, 40)
        if n == 1:
            lengths = str(total)
        else:
            lengths = "ragged:%d:%d:%d" % (n, rng.choice([0, 1, 5]), max(6, 2 * total // n))
        return dict(op=op, lengths=lengths, hk=hk, hv=min(hv, 32), dk=dk, dv=dv, dtype=dtype, pool=rng.random() < 0.5)
    tokens = _log_uniform(rng, 1, 12000)
    if op == "qk_gates":
        return dict(op=op, tokens=tokens, hk=hk, hv=hv, dk=rng.choice([32, 64, 128, 128]), dv=rng.choice([64, 128]), dtype=dtype)
    if op == "norm_gate":
        return dict(op=op, tokens=tokens, hv=hv, dv=rng.choice([16, 64, 128, 128]), dtype=dtype, act=rng.choice(["silu", "silu", "sigmoid"]))
    return dict(op=op, tokens=min(tokens, 6000), width=rng.choice([257, 768, 1000, 2048, 2560, 4096, 6144]), dtype=dtype,
                post=rng.random() < 0.5)


def _lengths(case):
    """The prompts' lengths; ragged ones are spread evenly over their range in a fixed shuffled order."""
    text = case["lengths"]
    if not text.startswith("ragged:"):
        return [int(x) for x in text.split(",")]
    n, low, high = (int(x) for x in text.split(":")[1:])
    step = 7 if n % 7 else 11
    return [low + (high - low) * ((i * step) % n) // max(1, n - 1) for i in range(n)]


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gates(gen, tokens, hv):
    """Log-decays from slow heads to fast ones and write strengths, as a model's own gates give them."""
    u = torch.rand(hv, device="cuda", generator=gen)
    rate = torch.exp(u * math.log(16.0))
    dt = torch.exp(torch.rand(hv, device="cuda", generator=gen) * math.log(100.0) + math.log(1e-3))
    bias = dt + torch.log(-torch.expm1(-dt))
    g = -rate * torch.nn.functional.softplus(torch.randn(tokens, hv, device="cuda", generator=gen) + bias)
    return g, torch.sigmoid(torch.randn(tokens, hv, device="cuda", generator=gen)), rate.log(), bias


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], _type(case)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = dict(case=dict(case), op=op)
    if op in ("prefill", "decode"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        if op == "prefill":
            lengths = _lengths(case)
            tokens, batch = sum(lengths), len(lengths)
        else:
            tokens = batch = case["batch"]
        unit = torch.nn.functional.normalize
        s["q"], s["k"] = unit(normal(tokens, hk, dk), dim=-1).to(dt), unit(normal(tokens, hk, dk), dim=-1).to(dt)
        # the values stay where the layer's fused projection left them: a slice of its rows
        rows = normal(tokens, 2 * hk * dk + hv * dv).to(dt)
        s["v"] = rows[:, 2 * hk * dk:].view(tokens, hv, dv)
        s["g"], s["beta"] = _gates(gen, tokens, hv)[:2]
        s["scale"] = dk ** -0.5
        if op == "prefill":
            s["lengths"] = lengths
            s["offsets"] = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
            if case["pool"]:
                states = batch + 5
                s["S"] = 0.1 * normal(states, hv, dv, dk)
                s["slots"] = torch.randperm(states, device="cuda", generator=gen)[:batch].to(torch.int32)
                s["fresh"] = (torch.arange(batch, device="cuda") % 3 != 1).to(torch.int32)
        else:
            states, dead = case["n_states"], case["dead"]
            s["S"] = 0.1 * normal(states, hv, dv, dk)
            s["slots"] = torch.randperm(states, device="cuda", generator=gen)[:batch].to(torch.int32)
            s["slots"][batch - dead:] = -1
            s["live"] = batch - dead
        return s
    tokens = case["tokens"]
    if op == "qk_gates":
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        rows = normal(tokens, 2 * hk * dk + hv * dv).to(dt)
        s["q"], s["k"] = rows[:, :hk * dk].view(tokens, hk, dk), rows[:, hk * dk:2 * hk * dk].view(tokens, hk, dk)
        ab = normal(tokens, 2 * hv).to(dt)
        s["a"], s["b"] = ab[:, :hv], ab[:, hv:]
        s["A_log"], s["dt_bias"] = _gates(gen, 1, hv)[2:]
    elif op == "norm_gate":
        hv, dv = case["hv"], case["dv"]
        s["o"] = (0.1 * normal(tokens, hv, dv)).to(dt)
        s["z"] = normal(tokens, hv, dv).to(dt)
        s["weight"] = (1.0 + 0.1 * normal(dv)).to(dt)
    else:
        width = case["width"]
        s["x"], s["y"] = (3.0 * normal(tokens, width)).to(dt), normal(tokens, width).to(dt)
        s["weight"] = (1.0 + 0.1 * normal(width)).to(dt)
        s["post"] = (1.0 + 0.1 * normal(width)).to(dt) if case["post"] else None
        s["scale"] = 0.7
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "qk_gates": _plain_qk_gates, "norm_gate": _plain_norm_gate,
            "residual_norm": _plain_residual_norm}[s["op"]](s)


def _run_own(s):
    from gated_delta_net_gb300 import binding as gb

    op = s["op"]
    if op == "prefill":
        if "S" in s:
            o, S = gb.gdn_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["offsets"], max(s["lengths"]), S0=s["S"],
                                  slots=s["slots"], fresh=s["fresh"], S_new=s["S"], scale=s["scale"])
        else:
            o, S = gb.gdn_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["offsets"], max(s["lengths"]), scale=s["scale"])
        return {"o": o, "S": S}
    if op == "decode":
        o = gb.gdn_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], slots=s["slots"], scale=s["scale"])
        return {"o": o, "S": s["S"]}
    if op == "qk_gates":
        q, k, g, beta = gb.gdn_qk_gates(s["q"], s["k"], s["a"], s["b"], s["A_log"], s["dt_bias"], eps=EPS)
        return {"q": q, "k": k, "g": g, "beta": beta}
    if op == "norm_gate":
        return {"y": gb.gdn_norm_gate(s["o"], s["z"], s["weight"], eps=EPS, act=s["case"]["act"])}
    h, n = gb.gdn_residual_norm(s["x"], s["y"], s["weight"], scale=s["scale"], post_weight=s["post"], eps=EPS)
    return {"h": h, "n": n}


# the plain forms


def _plain_prefill(s):
    """The chunked form over prompts padded to one length: padded tokens have k = v = g = beta = 0 and change nothing."""
    case, lengths = s["case"], s["lengths"]
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    batch, tokens = len(lengths), sum(lengths)
    chunks = max(1, -(-max(lengths) // CHUNK))
    span = chunks * CHUNK
    at = torch.tensor([0] + lengths, device="cuda").cumsum(0)
    t = torch.arange(span, device="cuda")
    rows = at[:-1, None] + t
    inside = rows < at[1:, None]
    rows = torch.where(inside, rows, torch.full_like(rows, tokens)).reshape(-1)

    def laid_out(x, repeat):
        x = torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:], dtype=torch.float32)])[rows]
        x = x.view(batch, chunks, CHUNK, *x.shape[1:]).transpose(2, 3)
        return x.repeat_interleave(repeat, dim=2) if repeat > 1 else x

    q, k, v = laid_out(s["q"], hv // hk), laid_out(s["k"], hv // hk), laid_out(s["v"], 1)
    gam = laid_out(s["g"], 1).cumsum(-1)
    beta = laid_out(s["beta"], 1)
    lower = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    decay = torch.exp(torch.where(lower, gam[..., :, None] - gam[..., None, :], torch.full((), -math.inf, device="cuda")))
    x = (beta[..., None] * decay * (k @ k.mT)).tril(-1)
    y = decay * (q @ k.mT)
    inv = torch.eye(CHUNK, device="cuda").expand_as(x).contiguous()
    for i in range(1, CHUNK):
        inv[..., i, :i] = -(x[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    u0 = inv @ (beta[..., None] * v)
    w = inv @ ((beta * torch.exp(gam))[..., None] * k)
    qd = torch.exp(gam)[..., None] * q
    last = gam[..., -1:]
    kd = torch.exp(last - gam)[..., None] * k
    del v, x, inv, decay
    if "S" in s:
        slots = s["slots"].long()
        S = s["S"][slots] * (s["fresh"] == 0)[:, None, None, None]
    else:
        S = torch.zeros(batch, hv, dv, dk, device="cuda")
    o = torch.empty(batch, chunks, hv, CHUNK, dv, device="cuda")
    for c in range(chunks):
        u = u0[:, c] - w[:, c] @ S.mT
        o[:, c] = qd[:, c] @ S.mT + y[:, c] @ u
        S = torch.exp(last[:, c])[..., None] * S + u.mT @ kd[:, c]
    o = (s["scale"] * o).transpose(2, 3).reshape(batch, span, hv, dv)[inside].to(s["q"].dtype)
    if "S" in s:
        s["S"][slots] = S
        S = s["S"]
    return {"o": o, "S": S}


def _plain_decode(s):
    n, case = s["live"], s["case"]
    rep = case["hv"] // case["hk"]
    q, k = s["q"].float().repeat_interleave(rep, dim=1)[:n], s["k"].float().repeat_interleave(rep, dim=1)[:n]
    slots = s["slots"][:n].long()
    S = torch.exp(s["g"][:n])[..., None, None] * s["S"][slots]
    u = s["beta"][:n, :, None] * (s["v"][:n].float() - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., None] * k[:, :, None, :]
    o = torch.zeros(case["batch"], case["hv"], case["dv"], device="cuda")
    o[:n] = s["scale"] * (S * q[:, :, None, :]).sum(-1)
    s["S"][slots] = S
    return {"o": o.to(s["q"].dtype), "S": s["S"]}


def _plain_qk_gates(s):
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + EPS)
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + EPS)
    x = s["a"].float() + s["dt_bias"]
    g = -torch.exp(s["A_log"]) * (torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs())))
    beta = 1.0 / (1.0 + torch.exp(-s["b"].float()))
    return {"q": q.to(s["q"].dtype), "k": k.to(s["k"].dtype), "g": g, "beta": beta}


def _plain_norm_gate(s):
    o, z = s["o"].float(), s["z"].float()
    gate = 1.0 / (1.0 + torch.exp(-z))
    if s["case"]["act"] == "silu":
        gate = z * gate
    y = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"].float() * gate
    return {"y": y.to(s["o"].dtype)}


def _plain_residual_norm(s):
    x, y = s["x"].float(), s["y"].float()
    if s["post"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post"].float()
    h = x + s["scale"] * y
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    return {"h": h.to(s["x"].dtype), "n": n.to(s["x"].dtype)}


# the definitions in 64 bits


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = {n: x.double() for n, x in s.items() if torch.is_tensor(x) and x.is_floating_point()}
    if op == "qk_gates":
        norm = torch.linalg.vector_norm
        x = d["a"] + d["dt_bias"]
        return {"q": d["q"] / torch.sqrt(norm(d["q"], dim=-1, keepdim=True) ** 2 + EPS),
                "k": d["k"] / torch.sqrt(norm(d["k"], dim=-1, keepdim=True) ** 2 + EPS),
                "g": -d["A_log"].exp() * torch.logaddexp(x, torch.zeros_like(x)), "beta": torch.sigmoid(d["b"])}
    if op == "norm_gate":
        gate = torch.sigmoid(d["z"]) * (d["z"] if case["act"] == "silu" else 1.0)
        return {"y": d["o"] / torch.sqrt(d["o"].square().mean(-1, keepdim=True) + EPS) * d["weight"] * gate}
    if op == "residual_norm":
        y = d["y"]
        if s["post"] is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * d["post"]
        h = d["x"] + s["scale"] * y
        return {"h": h, "n": h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * d["weight"]}
    # the gated delta rule, one token after another; requests in order of length, so that the live ones are a prefix
    hk, hv = case["hk"], case["hv"]
    lengths = s["lengths"] if op == "prefill" else [1] * s["live"]
    if len(lengths) * hv * case["dk"] * case["dv"] * max(lengths) > 3e11:
        return None
    order = sorted(range(len(lengths)), key=lambda b: -lengths[b])
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    first = torch.tensor([starts[b] for b in order], device="cuda")
    o = torch.zeros(d["v"].shape, device="cuda", dtype=torch.float64)
    if "S" in d:
        slots = s["slots"].long()[torch.tensor(order, device="cuda")]
        S = d["S"][slots]
        if "fresh" in s:
            S[s["fresh"][torch.tensor(order, device="cuda")] != 0] = 0.0
    else:
        S = torch.zeros(len(lengths), hv, case["dv"], case["dk"], device="cuda", dtype=torch.float64)
    alpha = d["g"].exp()
    live = len(order)
    for t in range(max(lengths)):
        while live and lengths[order[live - 1]] <= t:
            live -= 1
        rows = first[:live] + t
        q, k = (d[n][rows].repeat_interleave(hv // hk, dim=1) for n in ("q", "k"))
        now = S[:live]
        now.mul_(alpha[rows][..., None, None])
        u = d["beta"][rows][..., None] * (d["v"][rows] - torch.einsum("bhvk,bhk->bhv", now, k))
        now.add_(u[..., None] * k[:, :, None, :])
        o[rows] = s["scale"] * torch.einsum("bhvk,bhk->bhv", now, q)
    if "S" in d:
        whole = d["S"].clone()
        whole[slots] = S
    else:
        whole = torch.empty_like(S)
        whole[torch.tensor(order, device="cuda")] = S
    return {"o": o, "S": whole}


def work(case):
    """Each input read once, each output written once; the rule's own multiplications and additions."""
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("prefill", "decode"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        state = 4 * hv * dv * dk
        if op == "prefill":
            lengths = _lengths(case)
            tokens = sum(lengths)
            read = sum(i % 3 == 1 for i in range(len(lengths))) if case["pool"] else 0
            states = (len(lengths) + read) * state
        else:
            tokens = case["batch"] - case["dead"]
            states = 2 * tokens * state
        row = e * (2 * hk * dk + 2 * hv * dv) + 8 * hv
        # S k, S q and u k^T at two operations an entry, and the decay of S
        return {"bytes": tokens * row + states, "flops": tokens * hv * 7 * dk * dv}
    tokens = case["tokens"]
    if op == "qk_gates":
        hk, hv, dk = case["hk"], case["hv"], case["dk"]
        return {"bytes": tokens * (4 * e * hk * dk + 2 * e * hv + 8 * hv), "flops": tokens * (8 * hk * dk + 16 * hv)}
    if op == "norm_gate":
        return {"bytes": 3 * e * tokens * case["hv"] * case["dv"], "flops": 12 * tokens * case["hv"] * case["dv"]}
    return {"bytes": 4 * e * tokens * case["width"], "flops": 10 * tokens * case["width"]}
