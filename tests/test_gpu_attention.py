"""GPU parity of the attention operators (gdn_attention.h) against their float64 definitions (oracle.attention).

Every pool is filled with NaN outside the slots that hold a request's tokens, and page tables with ids far outside the
pool behind a request's pages.

Tolerances, for an output o = sum_s p_s v_s and A = sum_s p_s |v_s|:
  fp32: a score is a sum of at most 256 products, whose roundings add up to about 16 times 2^-24 of |q| |k| scale (10 at
    most here), 2^-17 of p; the sums over up to 2^12 slots add 2^-18: 2^-15 A.
  bf16: besides that every p is rounded to bf16 before it is multiplied by v, 2^-8 of it, and o once more: 2^-8 |o| +
    (2^-8 + 2^-15) A.  fp32 outputs of bf16 tokens are not rounded a second time.
  what is appended: fp32 arithmetic of a norm over d <= 256 entries and two products, at most 2^-18 of |x_1| + |x_2|, and the
    rounding to bf16, 2^-8.
"""
import numpy as np
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from oracle import attention as OA

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FAR_PAGE = 1 << 29  # an id that no pool has


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_net_gb300 import build
    build.build()
    gb.lib()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


class Case:
    """A cache with lens[b] + counts[b] random tokens for each request, NaN elsewhere, and queries."""

    def __init__(self, seed, lens, counts, hq, hkv, d, page, dtype, layout="rows", pad=0, far=True):
        gen = torch.Generator().manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float32)  # noqa: E731
        self.lens_list, self.counts = list(lens), list(counts)
        needs = [-(-(max(n, 0) + c) // page) for n, c in zip(lens, counts)]
        self.n_pages = sum(needs) + 2
        order = torch.randperm(self.n_pages, generator=gen)
        table = torch.full((len(lens), max(needs) + 1), FAR_PAGE if far else 0, dtype=torch.int32)
        at = 0
        k = torch.full((self.n_pages, page, hkv, d), float("nan"))
        v = k.clone()
        for b, n in enumerate(needs):
            table[b, :n] = order[at:at + n]
            for i in range(n):
                rows = min(page, max(lens[b], 0) + counts[b] - i * page)
                k[order[at + i], :rows], v[order[at + i], :rows] = normal(rows, hkv, d), normal(rows, hkv, d)
            at += n
        self.table, self.lens = table.cuda(), ints(*lens)
        self.k, self.v = (self.laid_out(x, layout, dtype) for x in (k, v))
        if layout == "both":  # keys and values of a page side by side in one tensor
            whole = torch.stack([k, v], dim=1).to(dtype).cuda()
            self.k, self.v = whole[:, 0], whole[:, 1]
        T = sum(counts)
        rows = torch.full((T, hq * d + pad), float("nan"), dtype=dtype)
        rows[:, :hq * d] = 1.5 * normal(T, hq * d)
        rows = rows.cuda()
        self.q = rows[:, :hq * d].view(T, hq, d)
        self.off = offsets(counts)
        self.scale = d ** -0.5

    @staticmethod
    def laid_out(x, layout, dtype):
        x = x.to(dtype).cuda()
        if layout == "heads":  # heads before rows
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "odd":  # rows that do not start on 16 bytes
            wide = torch.full((*x.shape[:3], x.shape[3] + 3), float("nan"), dtype=dtype, device="cuda")
            wide[..., 1:-2] = x
            return wide[..., 1:-2]
        return x

    @property
    def cache(self):
        return self.k, self.v, self.table, self.lens

    def oracle(self, mask=None, decode=False):
        kc, vc, t, n = np.nan_to_num(f64(self.k)), np.nan_to_num(f64(self.v)), self.table.cpu().numpy(), self.lens_list
        a = (f64(self.q), kc), (t, n, None if decode else self.off.cpu().numpy(), None if mask is None else mask.cpu().numpy(), self.scale)
        return OA.attend(*a[0], vc, *a[1]), OA.attend(*a[0], np.abs(vc), *a[1])


def close(got, ref, A, dtype):
    p_bits = 2.0 ** -8 if dtype == BF else 0.0
    o_bits = 2.0 ** -8 if got.dtype == BF else 0.0
    got = f64(got)
    assert got.shape == ref.shape
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - (o_bits * np.abs(ref) * 1.01 + (p_bits + 2.0 ** -15) * A + 1e-30)
    assert float(over.max(initial=0.0)) <= 0, np.argwhere(over > 0)[:8].tolist()


def tree_masks(seed, counts, words=None, empty=()):
    """Random draft trees' masks [T, words] (a node hangs on one of the six before it), with some rows left empty."""
    rng = np.random.default_rng(seed)
    words = words or max(1, -(-max(counts) // 32))
    out = []
    for n in counts:
        seen = np.zeros((n, words * 32), dtype=bool)
        for i in range(n):
            if i and rng.random() > 0.1:
                seen[i] = seen[i - rng.integers(1, min(i, 6) + 1)]
            seen[i, i] = True
        out.append(seen)
    bits = np.concatenate(out) if out else np.zeros((0, words * 32), dtype=bool)
    for row in empty:
        bits[row] = False
    packed = (bits.reshape(len(bits), words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.from_numpy(packed.view(np.int32).copy()).cuda()


# ---------------------------------------------------------------------------------------------- single tokens

LENS = [[0], [1], [14], [15], [16], [30, 31, 32, 33], [62, 63, 64], [127, 128, 0, 1], [300, -1, 5, -1], [513, 2], [2000, 0, 900], [4095]]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_decode_lengths(lens, dtype):
    c = Case(1 + len(lens), lens, [1] * len(lens), 8, 2, 128, 16, dtype)
    st = gb.new_status()
    o = gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale, dev_status=st)
    gb.check_status(st)
    close(o, *c.oracle(decode=True), dtype)
    for b, n in enumerate(lens):
        assert n >= 0 or not np.any(f64(o[b]))


HEADS = [(1, 1, 16, 16), (3, 1, 32, 8), (4, 4, 64, 64), (16, 1, 64, 32), (20, 1, 128, 16), (14, 2, 128, 24), (40, 2, 32, 5),
         (4, 2, 256, 16), (16, 2, 256, 64), (24, 1, 256, 3), (12, 4, 128, 1), (6, 6, 128, 128), (33, 1, 16, 40), (8, 1, 128, 48)]


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("hq,hkv,d,page", HEADS)
def test_decode_heads_widths_pages_and_types(hq, hkv, d, page, dtype, out_dtype):
    c = Case(hq * d + page, [70, 0, 333], [1] * 3, hq, hkv, d, page, dtype)
    st = gb.new_status()
    o = gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale, out_dtype=out_dtype, dev_status=st)
    gb.check_status(st)
    assert o.dtype == out_dtype
    close(o, *c.oracle(decode=True), dtype)


LAYOUTS = [("rows", 0), ("heads", 0), ("both", 8), ("odd", 3), ("rows", 5)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout,pad", LAYOUTS)
def test_decode_layouts(layout, pad, dtype):
    c = Case(7, [200, 31], [1, 1], 8, 2, 128, 16, dtype, layout, pad)
    close(gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale), *c.oracle(decode=True), dtype)


@pytest.mark.parametrize("dtype,d,n", [(F32, 64, 20000), (BF, 128, 40001), (BF, 256, 20000), (BF, 64, 33000)])
def test_decode_long_cache_is_split_and_joined(dtype, d, n):
    c = Case(3, [n, 100], [1, 1], 4, 1, d, 64, dtype)
    o = gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale)
    close(o, *c.oracle(decode=True), dtype)
    for _ in range(3):
        assert torch.equal(o, gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", [0.0, -0.2, 5.0])
def test_decode_scales(scale, dtype):
    c = Case(9, [400, 17], [1, 1], 8, 2, 64, 16, dtype)
    c.scale = scale
    got = gb.gdn_kv_decode(c.q, *c.cache, scale=scale)
    ref, A = c.oracle(decode=True)
    if scale == 5.0:  # scores of about 100: their own rounding, 2^-24 of |q| |k| scale in every product, is 2^-15 of p
        assert np.max(np.abs(f64(got) - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * A)) <= 0
    else:
        close(got, ref, A, dtype)


def test_decode_of_many_requests():
    lens = [(i * 37) % 90 - 1 for i in range(700)]
    c = Case(10, lens, [1] * 700, 2, 1, 64, 16, BF)
    close(gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale), *c.oracle(decode=True), BF)


# ---------------------------------------------------------------------------------------------- several tokens

COUNTS = [([5], [0]), ([1], [40]), ([2, 3], [0, 300]), ([16, 1, 0, 7], [64, 0, 9, 500]), ([33, 64], [1000, 3]), ([128], [129]), ([127, 129, 1], [2, 260, 127]),
          ([256], [31]), ([100, 4], [-1, 50]), ([200, 250], [1500, 0])]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("counts,lens", COUNTS, ids=str)
def test_attend_lengths(counts, lens, tree, dtype):
    c = Case(sum(counts), lens, counts, 8, 2, 128, 16, dtype)
    mask = tree_masks(1, counts) if tree else None
    st = gb.new_status()
    o = gb.gdn_kv_attend(c.q, *c.cache, c.off, max(counts), anc_mask=mask, scale=c.scale, dev_status=st)
    gb.check_status(st)
    close(o, *c.oracle(mask), dtype)


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("hq,hkv,d,page", HEADS)
def test_attend_heads_widths_pages_and_types(hq, hkv, d, page, dtype, out_dtype):
    counts, lens = [37, 2, 70], [100, 40, 0]
    c = Case(hq + d + page, lens, counts, hq, hkv, d, page, dtype)
    for mask in (None, tree_masks(2, counts)):
        o = gb.gdn_kv_attend(c.q, *c.cache, c.off, 70, anc_mask=mask, scale=c.scale, out_dtype=out_dtype)
        close(o, *c.oracle(mask), dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout,pad", LAYOUTS)
def test_attend_layouts(layout, pad, dtype):
    counts = [90, 40]
    c = Case(8, [200, 31], counts, 8, 2, 128, 16, dtype, layout, pad)
    mask = tree_masks(3, counts, words=8)
    close(gb.gdn_kv_attend(c.q, *c.cache, c.off, 90, anc_mask=mask, scale=c.scale), *c.oracle(mask), dtype)


@pytest.mark.parametrize("dtype,hq,d,n,length", [(BF, 4, 128, 700, 333), (BF, 1, 64, 1500, 0), (BF, 8, 256, 300, 77), (BF, 32, 128, 64, 3000), (F32, 2, 64, 400, 100)])
def test_attend_prompts_and_long_caches(dtype, hq, d, n, length):
    c = Case(12, [length], [n], hq, 1, d, 64, dtype)
    o = gb.gdn_kv_attend(c.q, *c.cache, c.off, n, scale=c.scale)
    close(o, *c.oracle(), dtype)
    assert torch.equal(o, gb.gdn_kv_attend(c.q, *c.cache, c.off, n, scale=c.scale))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [2, 40])
def test_attend_rows_that_see_nothing_and_rows_behind_the_last(rows, dtype):
    counts, lens = [rows, 3], [0, 20]
    c = Case(13, lens, counts, 8, 2, 128, 16, dtype)
    mask = tree_masks(4, counts, empty=(0, rows - 1, rows + 1))
    q = torch.cat([c.q, c.q[:2]])
    out = torch.full_like(q, 7.0)
    got = gb.gdn_kv_attend(q, *c.cache, c.off, max(rows, 3), anc_mask=torch.cat([mask, mask[:2]]), scale=c.scale, out=out)
    assert got is out and torch.all(out[-2:] == 7.0)
    ref, A = c.oracle(mask)
    close(out[:-2], ref, A, dtype)
    assert not np.any(f64(out[0])) and not np.any(f64(out[rows - 1])) and np.any(f64(out[rows + 1]))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [3, 40, 130])
def test_what_is_not_seen_does_not_matter(n, value, where, dtype):
    # a new token of one request holds what is not finite: only the tokens that see it may differ
    c = Case(14, [50, 33], [n, n], 8, 2, 128, 16, dtype)
    mask = tree_masks(5, [n, n])
    for m in (mask, None):
        clean = gb.gdn_kv_attend(c.q, *c.cache, c.off, n, anc_mask=m, scale=c.scale)
        j = n // 2
        page, row = OA.slot(c.table.cpu().numpy(), 0, 50 + j, 16)
        pool = getattr(c, where)
        kept = pool[page, row].clone()
        pool[page, row, :, 5] = value
        got = gb.gdn_kv_attend(c.q, *c.cache, c.off, n, anc_mask=m, scale=c.scale)
        pool[page, row] = kept
        seen = OA.bits(mask.cpu().numpy(), n)[:, j] if m is not None else np.tril(np.ones((n, n), dtype=bool))[:, j].repeat(1)
        seen = np.concatenate([seen[:n], np.zeros(n, dtype=bool)])
        assert torch.equal(got[torch.from_numpy(~seen).cuda()], clean[torch.from_numpy(~seen).cuda()])
        if where == "v":  # (an infinite key may have no weight)
            assert not torch.any(torch.isfinite(got[torch.from_numpy(seen).cuda()][..., 5]))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_device_checks(dtype):
    c = Case(15, [40, 9, 20], [3, 20, 4], 8, 2, 128, 16, dtype)
    mask = tree_masks(6, c.counts)
    ref, A = c.oracle(mask)

    def run(off=c.off, most=20, table=c.table, lens=c.lens, m=mask):
        st, out = gb.new_status(), torch.full_like(c.q, 7.0)
        gb.gdn_kv_attend(c.q, c.k, c.v, table, lens, off, most, anc_mask=m, scale=c.scale, out=out, dev_status=st)
        return int(st.item()), out

    bits, out = run(most=19)
    assert bits == 4 and torch.all(out[3:23] == 7.0)
    close(out[:3], ref[:3], A[:3], dtype), close(out[23:], ref[23:], A[23:], dtype)
    bits, out = run(off=ints(0, 3, 2, 27))
    assert bits & 32 and torch.all(out[2:3] != 7.0)
    bits, out = run(off=ints(0, 3, 23, 28))
    assert bits == 32 and torch.all(out[23:] == 7.0)
    bits, out = run(lens=ints(40, 900, 20))
    assert bits == 256 and torch.all(out[3:23] == 7.0)
    bits, out = run(lens=ints(40, -5, 20))
    assert bits == 256 and torch.all(out[3:23] == 7.0)
    close(out[23:], ref[23:], A[23:], dtype)
    for wrong in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        bad = c.table.clone()
        bad[1, 0] = wrong
        bits, out = run(table=bad)
        assert bits == 256
        close(out[:3], ref[:3], A[:3], dtype), close(out[23:], ref[23:], A[23:], dtype)
    st = gb.new_status()
    one = Case(16, [5, 6], [1, 1], 8, 2, 128, 16, dtype)
    bad = one.table.clone()
    bad[0, 0] = one.n_pages
    gb.gdn_kv_decode(one.q, one.k, one.v, bad, one.lens, dev_status=st)
    assert int(st.item()) == 256


def test_offsets_past_32_bits():
    # page strides that put the last pages more than 2^32 elements away
    c = Case(17, [100, 60], [1, 40], 8, 2, 128, 16, BF, far=False)
    stride = (1 << 32) // (c.n_pages - 1) // 64 * 64 + 64
    whole = [torch.empty(stride * (c.n_pages - 1) + 16 * 2 * 128, dtype=BF, device="cuda") for _ in range(2)]
    far = [w.as_strided((c.n_pages, 16, 2, 128), (stride, 256, 128, 1)) for w in whole]
    for f, x in zip(far, (c.k, c.v)):
        f.copy_(x)
    mask = tree_masks(7, [1, 40])
    want = gb.gdn_kv_attend(c.q, *c.cache, c.off, 40, anc_mask=mask, scale=c.scale)
    got = gb.gdn_kv_attend(c.q, *far, c.table, c.lens, c.off, 40, anc_mask=mask, scale=c.scale)
    assert torch.equal(got, want)
    q = c.q[:2].contiguous()
    assert torch.equal(gb.gdn_kv_decode(q, *far, c.table, c.lens, scale=c.scale), gb.gdn_kv_decode(q, *c.cache, scale=c.scale))
    gb.gdn_kv_append(None, c.k[0, :1].contiguous(), c.v[0, :1].contiguous(), *far, c.table[:1], c.lens[:1])
    page, row = OA.slot(c.table.cpu().numpy(), 0, 100, 16)
    assert torch.equal(far[0][page, row], c.k[0, 0]) and torch.equal(far[1][page, row], c.v[0, 0])


# ---------------------------------------------------------------------------------------------- streams, graphs, workspaces


@pytest.mark.parametrize("dtype", [F32, BF])
def test_graph_replays_with_other_lengths(dtype):
    c = Case(18, [3000, 700, 0], [1] * 3, 8, 1, 128, 16, dtype)
    tree = Case(19, [900, 30], [20, 50], 8, 1, 128, 16, dtype)
    mask = tree_masks(8, [20, 50])
    run = lambda: (gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale),  # noqa: E731
                   gb.gdn_kv_attend(tree.q, *tree.cache, tree.off, 50, anc_mask=mask, scale=tree.scale))
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for lens, lens2 in (([3000, 700, 0], [900, 30]), ([10, 690, -1], [5, 0]), ([2999, 1, 0], [899, 12])):
        c.lens.copy_(ints(*lens)), tree.lens.copy_(ints(*lens2))
        c.lens_list, tree.lens_list = lens, lens2
        g.replay()
        torch.cuda.synchronize()
        close(got[0], *c.oracle(decode=True), dtype)
        close(got[1], *tree.oracle(mask), dtype)


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 1, 64), (8, 1, 256), (32, 1, 16)])
def test_attend_of_many_requests(hq, hkv, d):
    # more requests than a block has threads, some empty, some not in use
    counts = [(i * 7) % 6 for i in range(900)]
    lens = [(i * 53) % 70 - 1 for i in range(900)]
    c = Case(41, lens, counts, hq, hkv, d, 16, BF)
    for mask in (None, tree_masks(9, counts)):
        o = gb.gdn_kv_attend(c.q, *c.cache, c.off, 5, anc_mask=mask, scale=c.scale)
        close(o, *c.oracle(mask), BF)


@pytest.mark.parametrize("dtype,d,lens,counts", [(BF, 128, [5000, 4000, 100], [3, 3, 2]), (BF, 64, [3000, 2000], [2, 40]), (F32, 64, [3000, 900], [2, 3]),
                                                 (BF, 128, [900, 30], [300, 20]), (BF, 256, [2500, 60], [40, 9])])
def test_attend_parts_of_trees_are_joined(dtype, d, lens, counts):
    # few items, long caches: most of them are cut, inside their committed slots and inside the new ones
    c = Case(42, lens, counts, 8, 2, d, 16, dtype)
    mask = tree_masks(10, counts)
    for m in (mask, None):
        o = gb.gdn_kv_attend(c.q, *c.cache, c.off, max(counts), anc_mask=m, scale=c.scale)
        close(o, *c.oracle(m), dtype)


def test_negative_and_zero_scales_of_several_tokens():
    c = Case(43, [300, 20], [40, 30], 8, 2, 128, 16, BF)
    for scale in (-0.1, 0.0):
        c.scale = scale
        close(gb.gdn_kv_attend(c.q, *c.cache, c.off, 40, scale=scale), *c.oracle(), BF)


def test_memory_of_a_dropped_result_on_another_stream():
    # what a call on the side stream returned goes back to the allocator while the call may still write it
    c = Case(44, [9000, 300], [1, 1], 8, 1, 128, 16, BF)
    ref = gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for _ in range(3):
            gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale, stream=side)
        ones = torch.ones(2, 8, 128, dtype=BF, device="cuda")
        got = gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, ref) and np.all(ones.float().cpu().numpy() == 1.0)


def test_append_then_attend_back_to_back():
    # the kernels may take their places while the one before ends: what it wrote is seen
    c = Case(45, [700, 90], [20, 9], 8, 2, 128, 16, BF)
    k, v = torch.randn(29, 2, 128, device="cuda").to(BF), torch.randn(29, 2, 128, device="cuda").to(BF)
    angles = table_of_angles(800, 64)
    mask = tree_masks(11, [20, 9])
    want = None
    for i in range(30):
        q = gb.gdn_kv_append(c.q, k, v, *c.cache, token_offsets=c.off, cos_sin=angles)
        o = gb.gdn_kv_attend(q, *c.cache, c.off, 20, anc_mask=mask, scale=c.scale)
        d = gb.gdn_kv_decode(q[:2].contiguous(), *c.cache, scale=c.scale)
        # another token's keys in between, so that a stale read shows
        gb.gdn_kv_append(None, v, k, *c.cache, token_offsets=c.off, cos_sin=angles)
        if want is None:
            torch.cuda.synchronize()
            want = o.clone(), d.clone()
        assert torch.equal(o, want[0]) and torch.equal(d, want[1])


def test_a_wait_that_runs_out_is_reported_and_changes_nothing():
    c = Case(46, [700, 90], [20, 40], 8, 2, 128, 16, BF)
    run = lambda st: gb.gdn_kv_attend(c.q, *c.cache, c.off, 40, scale=c.scale, dev_status=st)  # noqa: E731
    want = run(None)
    st = gb.new_status()
    gb.gdn_test_set_wait_probe(64)
    try:
        got = run(st)
    finally:
        gb.gdn_test_set_wait_probe(0)
    assert int(st.item()) == 16 and torch.equal(got, want)
    st = gb.new_status()
    assert torch.equal(run(st), want) and int(st.item()) == 0


def test_two_streams_at_once():
    cs = [Case(20 + i, [9000, 500], [1, 1], 8, 1, 128, 16, BF) for i in range(2)]
    refs = []
    for c in cs:
        refs.append(gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale))
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        here = [gb.gdn_kv_decode(cs[0].q, *cs[0].cache, scale=cs[0].scale) for _ in range(3)]
        there = [gb.gdn_kv_decode(cs[1].q, *cs[1].cache, scale=cs[1].scale, stream=side) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, refs[0]) for x in here) and all(torch.equal(x, refs[1]) for x in there)


def test_workspace_of_the_callers():
    c = Case(22, [5000, 3], [1, 1], 8, 1, 128, 16, BF)
    need = gb.gdn_kv_attend_workspace(c.q, c.k, c.v, c.table, decode=True)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    ref = gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale)
    for _ in range(2):
        assert torch.equal(gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale, workspace=ws), ref)
    with pytest.raises(gb.GdnError):
        gb.gdn_kv_decode(c.q, *c.cache, workspace=ws[:need - 1])


def test_refusals_of_the_binding():
    c = Case(23, [20], [1], 8, 2, 128, 16, BF)
    decode = lambda **kw: gb.gdn_kv_decode(**{**dict(q=c.q, k_cache=c.k, v_cache=c.v, page_table=c.table, lens=c.lens), **kw})  # noqa: E731
    decode()
    for kw in (dict(q=c.q.cpu()), dict(k_cache=c.k.float()), dict(v_cache=c.v.cpu()), dict(page_table=c.table.long()), dict(lens=c.lens.cpu()),
               dict(q=c.q.half())):
        with pytest.raises(TypeError):
            decode(**kw)
    for kw in (dict(v_cache=c.v[:-1]), dict(v_cache=c.v.transpose(1, 2).contiguous().transpose(1, 2)), dict(page_table=c.table[0]),
               dict(lens=c.lens.repeat(2)), dict(q=c.q.repeat(2, 1, 1)), dict(q=c.q[..., :64].contiguous())):
        with pytest.raises(ValueError):
            decode(**kw)
    with pytest.raises(gb.GdnError):
        decode(q=c.q[:, :3].contiguous())
    with pytest.raises(gb.GdnError):
        decode(scale=float("inf"))


# ---------------------------------------------------------------------------------------------- append and commit


def table_of_angles(positions, rot):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], axis=1)).float().cuda()


def near(got, ref, scale, dtype):
    got = f64(got)
    bits = 2.0 ** -8 if dtype == BF else 0.0
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.all(np.abs(got - ref)[ok] <= (bits * 1.01 * np.abs(ref) + 2.0 ** -18 * scale)[ok] + 1e-30)


APPENDS = [(8, 2, 128, 128, 16), (4, 4, 64, 16, 8), (16, 1, 256, 64, 64), (3, 1, 32, 8, 5), (2, 2, 16, 16, 1), (5, 5, 128, 0, 24), (8, 8, 128, 20, 16), (1, 1, 256, 256, 128),
           (6, 2, 32, 32, 16), (8, 2, 64, 2, 16)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved,norm,layout,pad", [(False, False, "rows", 0), (True, True, "heads", 8), (False, True, "both", 0), (False, True, "odd", 3),
                                                         (True, False, "odd", 1)])
@pytest.mark.parametrize("hq,hkv,d,rot,page", APPENDS)
def test_append(hq, hkv, d, rot, page, interleaved, norm, layout, pad, dtype):
    counts, lens = [5, 0, 1, 37, 2], [0, 12, 100, 15, -1]
    c = Case(d + rot, lens, counts, hq, hkv, d, page, dtype, layout, pad)
    T = sum(counts)
    gen = torch.Generator().manual_seed(3)
    rows = torch.randn(T, (hq + 2 * hkv) * d + pad, generator=gen).to(dtype).cuda()
    q, k, v = (rows[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    angles = table_of_angles(140, rot) if rot else None
    w = [(1 + 0.2 * torch.randn(d, generator=gen)).to(F32 if hq % 2 else dtype).cuda() if norm else None for _ in range(2)]
    depth = torch.cat([torch.arange(n) // 2 + 1 for n in counts]).to(torch.int32).cuda() if norm else None
    before = f64(c.k), f64(c.v)
    st = gb.new_status()
    out = torch.full((T, hq, d), float("nan"), dtype=dtype, device="cuda")
    got = gb.gdn_kv_append(q, k, v, *c.cache, token_offsets=c.off, depth=depth, cos_sin=angles, interleaved=interleaved, q_weight=w[0],
                           k_weight=w[1], q_out=out, dev_status=st)
    gb.check_status(st)
    assert got is out
    n = lambda x: None if x is None else x.cpu().numpy() if x.dtype == torch.int32 else f64(x)  # noqa: E731
    args = (n(c.table), lens, n(c.off), n(depth), n(angles), interleaved)
    rq, rk, rv = OA.append(f64(q), f64(k), f64(v), *before, *args, n(w[0]), n(w[1]))
    near(out, rq, np.max(np.abs(np.nan_to_num(rq)), axis=-1, keepdims=True) * 2, dtype)
    near(c.k, rk, np.nanmax(np.abs(rk)) * 2, dtype)
    assert np.array_equal(f64(c.v), rv, equal_nan=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_append_single_tokens_in_place_and_keys_only(dtype):
    lens = [3, -1, 0, 40]
    c = Case(30, lens, [1] * 4, 4, 2, 64, 16, dtype)
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(4, h, 64, generator=gen).to(dtype).cuda() for h in (4, 2, 2))
    angles = table_of_angles(41, 64)
    ref = OA.append(f64(q), f64(k), f64(v), f64(c.k), f64(c.v), c.table.cpu().numpy(), lens, cos_sin=f64(angles))
    again = Case(30, lens, [1] * 4, 4, 2, 64, 16, dtype)
    untouched = f64(q[1])
    got = gb.gdn_kv_append(q, k, v, *c.cache, cos_sin=angles, q_out=q)
    assert got is q and np.array_equal(f64(q[1]), untouched)
    rq = ref[0].copy()
    rq[1] = untouched
    near(q, rq, np.max(np.abs(rq)) * 2, dtype)
    near(c.k, ref[1], 8.0, dtype)
    assert gb.gdn_kv_append(None, k, v, *again.cache, cos_sin=angles) is None
    assert torch.equal(again.k.nan_to_num(9.0), c.k.nan_to_num(9.0)) and torch.equal(again.v.nan_to_num(9.0), c.v.nan_to_num(9.0))


def test_append_device_checks():
    def run(lens=(3, 20), off=(0, 4, 6), positions=64, table=None, depth=None):
        c = Case(31, [3, 20], [4, 2], 2, 1, 64, 16, BF)
        gen = torch.Generator().manual_seed(5)
        q, k, v = (torch.randn(6, h, 64, generator=gen).to(BF).cuda() for h in (2, 1, 1))
        before = c.k.clone(), c.v.clone()
        st, out = gb.new_status(), torch.full((6, 2, 64), 7.0, dtype=BF, device="cuda")
        t = c.table.clone()
        for at, x in (table or {}).items():
            t[at] = x
        gb.gdn_kv_append(q, k, v, c.k, c.v, t, ints(*lens), token_offsets=ints(*off), cos_sin=table_of_angles(positions, 64), q_out=out,
                         depth=None if depth is None else ints(*depth), dev_status=st)
        moved = [t for t in range(6) if not torch.all(out[t] == 7.0)]
        changed = int(((c.k != before[0]) & ~(c.k.isnan() & before[0].isnan())).any(-1).sum())
        return int(st.item()), moved, changed
    assert run() == (0, [0, 1, 2, 3, 4, 5], 6)
    assert run(positions=21) == (512, [0, 1, 2, 3, 4], 5)
    assert run(table={(1, 1): -1}) == (256, [0, 1, 2, 3], 4)
    assert run(table={(0, 0): 1 << 30}) == (256, [4, 5], 2)
    assert run(lens=(-2, 20)) == (256, [4, 5], 2)
    assert run(lens=(3, 1000)) == (256, [0, 1, 2, 3], 4)
    assert run(off=(0, 4, 7))[:2] == (32, [0, 1, 2, 3])
    assert run(off=(0, 4, 5)) == (0, [0, 1, 2, 3, 4], 5)
    assert run(off=(0, 5, 4))[0] == 32
    assert run(depth=(0, 1, 1, 2, 1, 2), lens=(0, 20)) == (512, [1, 2, 3, 4, 5], 5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hkv,d,page,layout", [(2, 128, 16, "rows"), (1, 64, 5, "heads"), (3, 256, 24, "both"), (2, 32, 1, "odd"), (1, 16, 64, "rows")])
def test_commit(hkv, d, page, layout, dtype):
    counts, lens = [12, 1, 0, 256, 30, 4], [5, 0, 7, 33, 100, -1]
    c = Case(d, lens, counts, hkv, hkv, d, page, dtype, layout)
    rng = np.random.default_rng(1)
    paths = [[0, 2, 3, 11], [0], [], list(range(0, 256, 1)), sorted(rng.choice(30, 11, replace=False).tolist()), [0, 1]]
    idx, po = np.concatenate(paths).astype(np.int32), np.concatenate([[0], np.cumsum([len(p) for p in paths])]).astype(np.int32)
    rk, rv, rl = OA.commit(f64(c.k), f64(c.v), c.table.cpu().numpy(), lens, po, idx)
    st = gb.new_status()
    new = gb.gdn_kv_commit(*c.cache, c.off, torch.from_numpy(po).cuda(), torch.from_numpy(idx).cuda(), dev_status=st)
    gb.check_status(st)
    assert np.array_equal(f64(c.k), rk, equal_nan=True) and np.array_equal(f64(c.v), rv, equal_nan=True)
    assert new.tolist() == rl.tolist()


def test_commit_device_checks():
    def run(path=((0, 2, 3), (1, 4)), lens=(10, 30), table=None, po=None, no=None):
        c = Case(33, [10, 30], [5, 6], 1, 1, 64, 16, BF)
        before = f64(c.k)
        t = c.table.clone()
        for at, x in (table or {}).items():
            t[at] = x
        idx = ints(*[j for p in path for j in p])
        st = gb.new_status()
        new = gb.gdn_kv_commit(c.k, c.v, t, ints(*lens), c.off if no is None else ints(*no), offsets([len(p) for p in path]) if po is None else ints(*po), idx, dev_status=st)
        mine = [sum(not np.array_equal(f64(c.k)[OA.slot(c.table.cpu().numpy(), b, s, 16)], before[OA.slot(c.table.cpu().numpy(), b, s, 16)], equal_nan=True)
                    for s in range([15, 36][b])) for b in range(2)]
        return int(st.item()), new.tolist(), mine
    assert run() == (0, [13, 32], [2, 2])
    assert run(path=((0, 5), (1, 4))) == (2, [10, 32], [0, 2])
    assert run(path=((2, 2), (1, 4))) == (2, [10, 32], [0, 2])
    assert run(path=((3, 1), (1, 4))) == (2, [10, 32], [0, 2])
    assert run(path=((-1, 1), (1, 4))) == (2, [10, 32], [0, 2])
    # (a path that does not ascend, at the end of the table: its targets lie past it)
    assert run(path=((5, 0, 1, 2, 3, 4), (1, 4)), lens=(59, 30), no=(0, 6, 12))[:2] == (258, [59, 32])
    assert run(table={(1, 2): 99}) == (256, [13, 30], [2, 0])
    assert run(lens=(10, 500)) == (256, [13, 500], [2, 0])
    assert run(lens=(10, -3)) == (256, [13, -3], [2, 0])
    assert run(lens=(10, -1)) == (0, [13, -1], [2, 0])
    assert run(po=(0, 3, 6)) == (32, [13, 30], [2, 0])
    assert run(no=(0, 5, 3)) == (32, [13, 30], [2, 0])
    assert run(path=((), ())) == (0, [10, 30], [0, 0])


def test_append_of_many_tokens():
    # past 16 tokens an SM a token has one warp
    counts = [1200, 0, 1400, 37]
    lens = [5, 9, 0, -1]
    for dtype, d, hq, hkv, rot, pad in ((BF, 64, 2, 1, 32, 0), (F32, 16, 3, 3, 16, 0), (BF, 256, 1, 1, 64, 3)):
        c = Case(34, lens, counts, hq, hkv, d, 16, dtype)
        T = sum(counts)
        gen = torch.Generator().manual_seed(6)
        rows = torch.randn(T, (hq + 2 * hkv) * d + pad, generator=gen).to(dtype).cuda()
        q, k, v = (rows[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        angles, w = table_of_angles(1500, rot), (1 + 0.2 * torch.randn(d, generator=gen)).to(dtype).cuda()
        before = f64(c.k), f64(c.v)
        st, out = gb.new_status(), torch.full((T, hq, d), float("nan"), dtype=dtype, device="cuda")
        gb.gdn_kv_append(q, k, v, *c.cache, token_offsets=c.off, cos_sin=angles, q_weight=w, k_weight=w, q_out=out, dev_status=st)
        gb.check_status(st)
        rq, rk, rv = OA.append(f64(q), f64(k), f64(v), *before, c.table.cpu().numpy(), lens, c.off.cpu().numpy(), None, f64(angles), False, f64(w), f64(w))
        near(out, rq, np.max(np.abs(np.nan_to_num(rq)), axis=-1, keepdims=True) * 2, dtype)
        near(c.k, rk, np.nanmax(np.abs(rk)) * 2, dtype)
        assert np.array_equal(f64(c.v), rv, equal_nan=True)


# ---------------------------------------------------------------------------------------------- together


def test_the_hybrid_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_serving.py")
    spec = importlib.util.spec_from_file_location("hybrid_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    # bf16 activations through two layers, four roundings of 2^-8 of the largest value each way
    assert module.run() <= 2.0 ** -5


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompts_drafts_commits_and_single_tokens_are_one_sequence(dtype):
    """A layer's tokens served in steps (prompts, a draft tree whose path is accepted, single tokens) and as one prompt."""
    hq, hkv, d, page, rot = 8, 2, 128, 16, 64
    prompt, accepted, singles = [70, 9], [5, 3], 4
    tree = [12, 7]
    gen = torch.Generator().manual_seed(40)
    lengths = [p + a + singles for p, a in zip(prompt, accepted)]
    toks = [[torch.randn(n, h, d, generator=gen).to(dtype).cuda() for h in (hq, hkv, hkv)] for n in lengths]
    angles = table_of_angles(200, rot)
    scale, st = d ** -0.5, gb.new_status()

    def fresh():
        table = torch.randperm(16, generator=gen).to(torch.int32).view(2, 8).cuda()
        return [torch.full((16, page, hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2)] + [table, ints(0, 0)]

    def prompts(cache, parts, counts):
        q, k, v = (torch.cat([x[i] for x in parts]) for i in range(3))
        q = gb.gdn_kv_append(q, k, v, *cache, token_offsets=offsets(counts), cos_sin=angles, dev_status=st)
        return gb.gdn_kv_attend(q, *cache, offsets(counts), max(counts), scale=scale, dev_status=st).split(counts)

    whole = prompts(fresh(), toks, lengths)

    cache = fresh()
    got = [list(prompts(cache, [[x[:p] for x in t] for t, p in zip(toks, prompt)], prompt))]
    cache[3] = ints(*prompt)
    # the draft: the accepted tokens are a path through a tree of other tokens
    paths = [[0, 2, 3, 7, 11], [1, 2, 6]]
    parents, nodes = [], []
    for b in range(2):
        parent = [-1] * tree[b]
        for a, n in zip(paths[b], paths[b][1:]):
            parent[n] = a
        x = [torch.randn(tree[b], h, d, generator=gen).to(dtype).cuda() for h in (hq, hkv, hkv)]
        for i in range(3):
            x[i][paths[b]] = toks[b][i][prompt[b]:prompt[b] + accepted[b]]
        for n in range(1, tree[b]):
            if n not in paths[b]:
                parent[n] = n - 1
        parents += parent
        nodes.append(x)
    no = offsets(tree)
    mask, depth = gb.gdn_tree_build_desc(ints(*parents), no, max(tree), dev_status=st)
    q, k, v = (torch.cat([x[i] for x in nodes]) for i in range(3))
    q = gb.gdn_kv_append(q, k, v, *cache, token_offsets=no, depth=depth, cos_sin=angles, dev_status=st)
    o = gb.gdn_kv_attend(q, *cache, no, max(tree), anc_mask=mask, scale=scale, dev_status=st).split(tree)
    got.append([o[b][paths[b]] for b in range(2)])
    cache[3] = gb.gdn_kv_commit(*cache, no, offsets(accepted), ints(*sum(paths, [])), dev_status=st)
    assert cache[3].tolist() == [p + a for p, a in zip(prompt, accepted)]
    for s in range(singles):
        x = [torch.stack([t[i][p + a + s] for t, p, a in zip(toks, prompt, accepted)]) for i in range(3)]
        q = gb.gdn_kv_append(*x, *cache, cos_sin=angles, dev_status=st)
        got.append(list(gb.gdn_kv_decode(q, *cache, scale=scale, dev_status=st).split(1)))
        cache[3] = cache[3] + 1
    gb.check_status(st)
    for b in range(2):
        steps = torch.cat([g[b] for g in got])
        # the same rows in other tiles: each is as near to the definition as close() asks, 2^-7 of values up to 4 apart
        assert float((steps.float() - whole[b].float()).abs().max()) <= (2.0 ** -4 if dtype == BF else 2.0 ** -13)
