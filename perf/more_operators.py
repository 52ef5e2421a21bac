"""What the attention operators of gated_delta_net_gb300 are measured on: the paged key-value cache of the attention
layers that stand between gated-delta-net layers.  New tokens are appended with the position rotation on the way,
single tokens, draft trees and prompts attend to the cache, and an accepted path is committed in it.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the end) or,
where `own` is true, calls the framework.  `exact` is the definition in 64 bits.  Slot s of request b is row
s % page_size of page page_table[b][s // page_size]; lens[b] tokens are committed, new tokens stand in the slots behind
them.  Batch and tree sizes are those of this repository's workloads (64 trees of 128 nodes); head counts, widths,
pages and lengths are generic.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0


def listed():
    return [
        # one user's next token, heads of 256 of which a quarter is rotated, queries and keys normed first
        dict(name="append_t1", op="append", batch=1, new="1:1", lens="4000:4000", dead=0, hq=16, hkv=2, d=256, rot=64, norm=True,
             interleaved=False, tree=False, page=64, dtype="bf16"),
        # a full serving batch padded to its graph's size: a token each, some rows not in use
        dict(name="append_b256", op="append", batch=256, new="1:1", lens="0:1500", dead=7, hq=32, hkv=4, d=128, rot=128, norm=False,
             interleaved=False, tree=False, page=16, dtype="bf16"),
        # a step's prompts, packed
        dict(name="append_prompts_16k", op="append", batch=40, new="20:800", lens="0:100", dead=0, hq=16, hkv=2, d=256, rot=64, norm=True,
             interleaved=False, tree=False, page=64, dtype="bf16"),
        # one user, a short conversation: latency
        dict(name="decode_b1", op="decode", batch=1, lens="700:700", dead=0, hq=32, hkv=8, d=128, page=16, dtype="bf16"),
        # one user, a very long document: only the split of its length fills the GPU
        dict(name="decode_b1_long", op="decode", batch=1, lens="131071:131071", dead=0, hq=32, hkv=4, d=128, page=64, dtype="bf16"),
        # a full serving batch with conversations of every length
        dict(name="decode_b128_ragged", op="decode", batch=128, lens="10:6000", dead=5, hq=32, hkv=8, d=128, page=16, dtype="bf16"),
        # the 32-bit form, as a numerics check of a model runs it; pages of no power of two
        dict(name="decode_f32_b5", op="decode", batch=5, lens="0:2500", dead=0, hq=12, hkv=4, d=64, page=24, dtype="f32"),
        # small draft trees for a few users
        dict(name="attend_drafts_b8", op="attend", batch=8, new="6:16", lens="500:6000", tree=True, hq=32, hkv=8, d=128, page=16, dtype="bf16"),
        # the serving batch of draft trees
        dict(name="attend_trees_b64_n128", op="attend", batch=64, new="128:128", lens="200:2200", tree=True, hq=32, hkv=8, d=128, page=32,
             dtype="bf16"),
        # a long prompt behind a shared prefix that is cached already
        dict(name="attend_prompt_8k", op="attend", batch=1, new="8192:8192", lens="777:777", tree=False, hq=32, hkv=8, d=128, page=64,
             dtype="bf16"),
        # one user's accepted draft
        dict(name="commit_b1", op="commit", batch=1, new="16:16", lens="900:900", hq=32, hkv=8, d=128, page=16, dtype="bf16"),
        # the serving batch's accepted drafts
        dict(name="commit_b64", op="commit", batch=64, new="128:128", lens="100:900", hq=32, hkv=8, d=128, page=32, dtype="bf16"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _range(low, high, batch):
    """A range of sizes; a single request has its upper end."""
    return "%d:%d" % (low if batch > 1 else high, high)


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "attend", "attend", "commit"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 7, 8])
    d = rng.choice([32, 64, 128, 128, 128, 256])
    case = dict(op=op, hq=hq, hkv=hkv, d=d, page=rng.choice([8, 16, 16, 24, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op == "append":
        batch = _log_uniform(rng, 1, 256)
        most = max(1, min(2 * _log_uniform(rng, 1, 400), 16000 // batch))
        case.update(batch=batch, new=_range(rng.choice([0, 1, 1]) if most > 1 else 1, most, batch),
                    lens=_range(0, _log_uniform(rng, 1, 2000), batch), dead=rng.randint(0, batch // 8) if most == 1 else 0,
                    rot=rng.choice([d, d, d // 2, d // 4]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.3,
                    tree=1 < most <= 256 and rng.random() < 0.4)
    elif op == "decode":
        batch = _log_uniform(rng, 1, 128)
        # at most as many bytes as 128 conversations of 3000 tokens, 8 heads of width 128 in 16 bits
        most = int(128 * 6000 * 8 * 128 * 2 / (batch * hkv * d * (2 if case["dtype"] == "bf16" else 4)))
        case.update(batch=batch, lens=_range(rng.choice([0, 1, 100]), _log_uniform(rng, 120, min(131071, max(130, most))), batch),
                    dead=rng.randint(0, batch // 8))
    elif op == "attend":
        batch = _log_uniform(rng, 1, 64)
        tree = rng.random() < 0.7
        new = _log_uniform(rng, 2, 256 if tree else 4000)
        # at most 3e8 scores, a quarter of that in 32 bits
        keys = (3e8 if case["dtype"] == "bf16" else 0.75e8) / (batch * hq * new)
        length = _log_uniform(rng, 10, min(8000, max(20, keys)))
        if new + length > 2 * max(keys, 40):
            new = max(2, new // 8)
        case.update(batch=batch, new=_range(rng.choice([1, new]), new, batch), lens=_range(rng.choice([0, length]), length, batch), tree=tree)
    else:
        new, batch = _log_uniform(rng, 1, 256), _log_uniform(rng, 1, 64)
        case.update(batch=batch, new=_range(rng.choice([1, new]), new, batch), lens=_range(0, _log_uniform(rng, 1, 900), batch))
    return case


def _spread(text, n):
    """n whole numbers spread evenly over a range, in a fixed shuffled order."""
    low, high = (int(x) for x in text.split(":"))
    step = 7 if n % 7 else 11
    return [low + (high - low) * ((i * step) % n) // max(1, n - 1) for i in range(n)]


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _trees(counts, gen):
    """Draft trees as request-local parents: each node hangs on one of the four before it, so that depths grow with sizes."""
    most = max(counts)
    back = torch.randint(1, 5, (len(counts), most), generator=gen)
    at = torch.arange(most)
    parent = (at - back).clamp(min=0)
    parent[:, 0] = -1
    seen = torch.zeros(len(counts), most, most, dtype=torch.bool)
    every = torch.arange(len(counts))
    for i in range(most):
        if i:
            seen[:, i] = seen[every, parent[:, i]]
        seen[:, i, i] = True
    return seen


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    op, dt, batch, hq, hkv, d, page = (case[n] for n in ("op", "dtype", "batch", "hq", "hkv", "d", "page"))
    dt = _type(case)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    counts = _spread(case["new"], batch) if "new" in case else [1] * batch
    lens = _spread(case["lens"], batch)
    s = dict(case=dict(case), op=op, counts=counts, most=max(counts))
    needs = [-(-(n + c) // page) for n, c in zip(lens, counts)]
    n_pages = sum(needs) + 3
    order = torch.randperm(n_pages, generator=host).to(torch.int32)
    table = torch.full((batch, max(1, max(needs))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(needs):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table.cuda()
    s["k_cache"] = normal(n_pages, page, hkv, d).to(dt)
    s["v_cache"] = normal(n_pages, page, hkv, d).to(dt)
    live = batch - case.get("dead", 0)
    s["lens"] = torch.tensor(lens[:live] + [-1] * (batch - live), dtype=torch.int32, device="cuda")
    s["live"] = live
    s["offsets"] = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    tokens = sum(counts)
    if op == "append":
        # queries, keys and values stay where the layer's fused projection left them
        rows = normal(tokens, (hq + 2 * hkv) * d).to(dt)
        s["q"] = rows[:, :hq * d].view(tokens, hq, d)
        s["k"] = rows[:, hq * d:(hq + hkv) * d].view(tokens, hkv, d)
        s["v"] = rows[:, (hq + hkv) * d:].view(tokens, hkv, d)
        half = case["rot"] // 2
        angle = torch.arange(max(lens) + max(counts) + 1, device="cuda", dtype=torch.float64)[:, None] * BASE ** (
            -torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        s["q_weight"] = (1.0 + 0.1 * normal(d)).to(dt) if case["norm"] else None
        s["k_weight"] = (1.0 + 0.1 * normal(d)).to(dt) if case["norm"] else None
        s["single"] = case["new"] == "1:1"
        # a draft's nodes stand at their depth in the tree, which counts from one
        s["depth"] = None
        if case["tree"]:
            depth = _trees(counts, host).sum(-1).to(torch.int32)
            s["depth"] = torch.cat([depth[b, :c] for b, c in enumerate(counts)]).cuda()
    elif op == "decode":
        s["q"] = (1.5 * normal(batch, hq, d)).to(dt)
        s["scale"] = d ** -0.5
    elif op == "attend":
        s["q"] = (1.5 * normal(tokens, hq, d)).to(dt)
        s["scale"] = d ** -0.5
        s["mask"] = None
        if case["tree"]:
            words = -(-max(counts) // 32)
            seen = _trees(counts, host)
            bits = torch.zeros(batch, max(counts), words * 32, dtype=torch.int64)
            bits[:, :, :max(counts)] = seen
            packed = (bits.view(batch, -1, words, 32) << torch.arange(32)).sum(-1)
            packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
            s["mask"] = torch.cat([packed[b, :c] for b, c in enumerate(counts)]).contiguous().cuda()
    else:
        seen = _trees(counts, host)
        # the accepted path: that of a node of the tree's second half
        paths = [seen[b, min(c - 1, c // 2 + (c * 7 + b) % max(1, c // 2)), :c].nonzero().flatten() for b, c in enumerate(counts)]
        s["path"] = torch.cat(paths).to(torch.int32).cuda()
        s["path_offsets"] = torch.tensor([0] + [len(p) for p in paths]).cumsum(0).to(torch.int32).cuda()
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "decode": _plain_decode, "attend": _plain_attend, "commit": _plain_commit}[s["op"]](s)


def _run_own(s):
    from gated_delta_net_gb300 import binding as gb

    op, cache = s["op"], (s["k_cache"], s["v_cache"], s["table"], s["lens"])
    if op == "append":
        q = gb.gdn_kv_append(s["q"], s["k"], s["v"], *cache, token_offsets=None if s["single"] else s["offsets"], depth=s["depth"],
                             cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"], q_weight=s["q_weight"],
                             k_weight=s["k_weight"], eps=EPS)
        return {"q": q[:s["live"]] if s["single"] else q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "decode":
        return {"o": gb.gdn_kv_decode(s["q"], *cache, scale=s["scale"])}
    if op == "attend":
        return {"o": gb.gdn_kv_attend(s["q"], *cache, s["offsets"], s["most"], anc_mask=s["mask"], scale=s["scale"])}
    lens = gb.gdn_kv_commit(*cache, s["offsets"], s["path_offsets"], s["path"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": lens}


# the plain forms


def _slots(s, request, slot):
    """(page, row) of slots of requests."""
    page = s["case"]["page"]
    return s["table"][request, slot // page].long(), slot % page


def _of_tokens(offsets, tokens):
    """(request, place in it) of every packed token."""
    t = torch.arange(tokens, device="cuda")
    request = torch.searchsorted(offsets[1:].long(), t, right=True)
    return request, t - offsets[request].long()


def _plain_append(s):
    case = s["case"]
    request, place = _of_tokens(s["offsets"], s["q"].shape[0])
    if s["single"]:
        request, place = request[:s["live"]], place[:s["live"]]
    n = request.shape[0]
    start = s["lens"][request].long()
    position = start + (place if s["depth"] is None else s["depth"].long() - 1)
    rot = case["rot"]
    cos, sin = s["cos_sin"][position][:, None].split(rot // 2, dim=-1)

    def turned(x, weight):
        x = x[:n].float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([y, x[..., rot:]], dim=-1)

    page, row = _slots(s, request, start + place)
    s["k_cache"][page, row] = turned(s["k"], s["k_weight"]).to(s["k"].dtype)
    s["v_cache"][page, row] = s["v"][:n]
    return {"q": turned(s["q"], s["q_weight"]).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(s, cache, slots):
    """[B, Hkv, slots, d] in 32 bits: every request's first slots (any value where it has none)."""
    page = s["case"]["page"]
    table = s["table"].clamp(min=0).long()
    pages = cache[table].flatten(1, 2)
    if slots > pages.shape[1]:
        slots = pages.shape[1]
    return pages[:, :slots].transpose(1, 2).float()


def _softmax_product(scores, seen, v):
    scores = torch.where(seen, scores, torch.full((), -math.inf, device="cuda"))
    scores = scores - scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores)
    del scores
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.clamp(min=1e-30)


def _plain_decode(s):
    case = s["case"]
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    slots = s["table"].shape[1] * case["page"]
    k, v = _gathered(s, s["k_cache"], slots), _gathered(s, s["v_cache"], slots)
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    seen = (torch.arange(slots, device="cuda") <= s["lens"][:, None]) & (s["lens"] >= 0)[:, None]
    o = _softmax_product(s["scale"] * (q @ k.mT), seen[:, None, None], v)
    return {"o": o.reshape(b, hq, d).to(s["q"].dtype)}


def _plain_attend(s):
    case = s["case"]
    b, hq, hkv, d, most = case["batch"], case["hq"], case["hkv"], case["d"], s["most"]
    slots = s["table"].shape[1] * case["page"]
    k, v = _gathered(s, s["k_cache"], slots), _gathered(s, s["v_cache"], slots)
    tokens = s["q"].shape[0]
    request, place = _of_tokens(s["offsets"], tokens)
    q = torch.zeros(b, most, hq, d, device="cuda")
    q[request, place] = s["q"].float()
    q = q.view(b, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    slot, lens = torch.arange(slots, device="cuda"), s["lens"].long()
    new = slot[None] - lens[:, None]
    if s["mask"] is None:
        seen = new[:, None, :] <= torch.arange(most, device="cuda")[None, :, None]
    else:
        words = torch.zeros(b, most, s["mask"].shape[1], dtype=torch.int32, device="cuda")
        words[request, place] = s["mask"]
        at = new.clamp(min=0, max=32 * words.shape[2] - 1)
        word = torch.gather(words, 2, (at // 32)[:, None].expand(b, most, slots))
        seen = ((word >> (at % 32)[:, None]) & 1).bool() & (new >= 0)[:, None] & (new < 32 * words.shape[2])[:, None]
        seen = seen | (new < 0)[:, None]
    scores = s["scale"] * (q.flatten(2, 3) @ k.mT)
    seen = seen[:, None, None].expand(b, 1, hq // hkv, most, slots).flatten(2, 3)
    o = _softmax_product(scores, seen, v)
    del scores
    o = o.view(b, hkv, hq // hkv, most, d).permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)
    return {"o": o[request, place].to(s["q"].dtype)}


def _plain_commit(s):
    request, place = _of_tokens(s["path_offsets"], s["path"].shape[0])
    lens = s["lens"].long()[request]
    source, target = _slots(s, request, lens + s["path"].long()), _slots(s, request, lens + place)
    s["k_cache"][target] = s["k_cache"][source]
    s["v_cache"][target] = s["v_cache"][source]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["lens"] + s["path_offsets"].diff()}


# the definitions in 64 bits, a request after another


def exact(case, seed):
    s, op, page, hkv = prepare(case, seed), case["op"], case["page"], case["hkv"]
    group = case["hq"] // hkv
    table, lens, ends = s["table"].tolist(), s["lens"].tolist(), s["offsets"].tolist()

    def where(b, slots):
        pages = s["table"][b].long()
        return pages[slots // page], slots % page

    if op == "commit":
        k, v, at = s["k_cache"].double(), s["v_cache"].double(), s["path_offsets"].tolist()
        for b in range(case["batch"]):
            path = s["path"][at[b]:at[b + 1]].long()
            old, new = where(b, lens[b] + path), where(b, lens[b] + torch.arange(len(path), device="cuda"))
            k[new], v[new] = k[old], v[old]
        return {"k_cache": k, "v_cache": v, "lens": None}
    if op == "append":
        k, v, rot = s["k_cache"].double(), s["v_cache"].double(), case["rot"]
        half = rot // 2
        first = torch.arange(0, rot, 2) if case["interleaved"] else torch.arange(half)
        second = first + (1 if case["interleaved"] else half)

        def turned(x, w, position):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
            turn = torch.complex(s["cos_sin"][position, :half].double(), s["cos_sin"][position, half:].double())
            z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        out = []
        for b in range(s["live"]):
            rows = slice(ends[b], ends[b + 1])
            place = torch.arange(ends[b + 1] - ends[b], device="cuda")
            position = lens[b] + (place if s["depth"] is None else s["depth"][rows].long() - 1)
            out.append(turned(s["q"][rows], s["q_weight"], position))
            new = where(b, lens[b] + place)
            k[new], v[new] = turned(s["k"][rows], s["k_weight"], position), s["v"][rows].double()
        return {"q": torch.cat(out), "k_cache": k, "v_cache": v}
    o = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    for b in range(s["live"]):
        n = 1 if op == "decode" else ends[b + 1] - ends[b]
        if not n:
            continue
        rows = slice(b, b + 1) if op == "decode" else slice(ends[b], ends[b + 1])
        old = where(b, torch.arange(lens[b] + n, device="cuda"))
        k, v = s["k_cache"][old].double(), s["v_cache"][old].double()
        if s.get("mask") is None:
            seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            column = torch.arange(n, device="cuda")
            seen = (s["mask"][rows][:, column // 32] >> (column % 32) & 1) != 0
        hidden = torch.zeros(n, lens[b] + n, dtype=torch.float64, device="cuda")
        hidden[:, lens[b]:].masked_fill_(~seen, -math.inf)
        for h in range(hkv):
            for g in range(h * group, (h + 1) * group):
                p = torch.softmax(s["scale"] * s["q"][rows, g].double() @ k[:, h].T + hidden, dim=-1)
                o[rows, g] = p @ v[:, h]
    return {"o": o}


def work(case):
    """Each input read once, each output written once; two products of two operations an entry for every visible key."""
    op, e, batch, hq, hkv, d = case["op"], 2 if case["dtype"] == "bf16" else 4, case["batch"], case["hq"], case["hkv"], case["d"]
    lens = _spread(case["lens"], batch)
    counts = _spread(case["new"], batch) if "new" in case else [1] * batch
    live = batch - case.get("dead", 0)
    if op == "append":
        tokens = sum(counts[:live])
        return {"bytes": tokens * (e * d * (2 * hq + 4 * hkv) + 4 * case["rot"]),
                "flops": tokens * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if op == "commit":
        # paths: a node in two of the trees' later half
        moved = sum(max(1, (3 * c // 4) * 2 // 5) for c in counts)
        return {"bytes": 4 * e * moved * hkv * d, "flops": 0}
    keys = sum(n + c for n, c in zip(lens[:live], counts))
    rows = live if op == "decode" else sum(counts)
    if op == "decode":
        pairs = keys
    elif case["tree"]:
        # a node sees the committed tokens and its path, about two fifths of the nodes before it
        pairs = sum(c * n + c * (c + 1) // 5 for n, c in zip(lens, counts))
    else:
        pairs = sum(c * n + c * (c + 1) // 2 for n, c in zip(lens, counts))
    return {"bytes": 2 * e * hkv * d * keys + 2 * e * rows * hq * d, "flops": 4 * hq * d * pairs}
