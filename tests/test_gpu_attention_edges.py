"""Edges of the attention operators (gdn_attention.h): what is not finite, and where it may not reach.

Cases and tolerances are those of test_gpu_attention; what has to be zero, NaN or unchanged is so exactly.
"""
import numpy as np
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from oracle import attention as OA
from tests.test_gpu_attention import BF, F32, Case, close, f64, tree_masks

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_net_gb300 import build
    build.build()
    gb.lib()


def attend(c, mask=None, **kw):
    return gb.gdn_kv_attend(c.q, *c.cache, c.off, max(c.counts), anc_mask=mask, scale=c.scale, **kw)


def own_slot(c, b, i):
    """Page and row of new token i of request b."""
    return OA.slot(c.table.cpu().numpy(), b, max(c.lens_list[b], 0) + i, c.k.shape[1])


# query heads, key-value heads, width, the second request's tokens: few rows, and more than 16 (in one token, or beside it)
KINDS = [(8, 2, 128, 1), (4, 1, 16, 3), (8, 2, 256, 2), (8, 2, 128, 40), (8, 2, 64, 300), (8, 2, 256, 40), (32, 1, 128, 1), (128, 1, 64, 1)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("length", [0, 50, 3000])
@pytest.mark.parametrize("hq,hkv,d,other", KINDS)
def test_a_single_token_that_does_not_see_itself(hq, hkv, d, other, length, where, dtype):
    c = Case(60, [length, 20], [1, other], hq, hkv, d, 16, dtype)
    mask = tree_masks(1, c.counts, empty=(0,))
    page, row = own_slot(c, 0, 0)
    outs = []
    for value in (1.0, NAN, INF, -INF):
        getattr(c, where)[page, row] = value
        outs.append(attend(c, mask))
    assert torch.isfinite(outs[0]).all() and (length > 0 or not torch.any(outs[0][0]))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def definition(c, mask=None, decode=False):
    """The definition with what is infinite (slots that hold nothing are not seen)."""
    k, v = (np.nan_to_num(f64(x), nan=0.0, posinf=np.inf, neginf=-np.inf) for x in (c.k, c.v))
    a = (c.table.cpu().numpy(), c.lens_list, None if decode else c.off.cpu().numpy(), None if mask is None else mask.cpu().numpy(), c.scale)
    with np.errstate(invalid="ignore"):
        return OA.attend(f64(c.q), k, v, *a), OA.attend(f64(c.q), k, np.abs(v), *a)


def same_but_where_nan(got, ref, A, dtype):
    bad = np.isnan(ref)
    assert np.array_equal(np.isnan(f64(got)), bad)
    close(torch.where(torch.from_numpy(bad).cuda(), torch.zeros_like(got), got), np.where(bad, 0.0, ref), np.where(bad, 0.0, A), dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("hq,hkv,d,lens,counts", [(8, 2, 128, [0, 9], [1, 2]), (8, 2, 128, [0, 9], [40, 3]), (8, 2, 64, [0, 0], [130, 2]), (4, 1, 256, [0, 30], [70, 1]),
                                                  (4, 1, 32, [0, 3], [20, 4])])
def test_an_infinite_entry_of_the_first_key(hq, hkv, d, lens, counts, value, dtype):
    # its scores are infinite, of either sign: the first token sees nothing else, the softmax is NaN; the later tokens' heads
    # with a negative one give it no weight
    c = Case(61, lens, counts, hq, hkv, d, 16, dtype)
    for b in range(2):
        c.k[int(c.table[b, 0]), 0, :, 5] = value
    for mask in (None, tree_masks(2, counts)):
        ref, A = definition(c, mask)
        assert np.isnan(ref[0]).all() and (counts[0] < 20 or np.isfinite(ref[19]).any())
        same_but_where_nan(attend(c, mask), ref, A, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hq,hkv,d,lens,counts", [(8, 2, 128, [20, 0], [3, 4]), (8, 1, 128, [0, 700], [200, 60]), (4, 1, 64, [0, 40], [300, 2]), (4, 1, 256, [0, 3000], [130, 60]),
                                                  (8, 2, 128, [3000, 0], [2, 2])])
def test_infinite_scores_in_every_slot(hq, hkv, d, lens, counts, dtype):
    # NaN for the tokens that see a slot, zeros for those that see none, in items that are cut and joined too
    c = Case(62, lens, counts, hq, hkv, d, 16, dtype)
    c.k[..., 5] = -INF
    empty = [sum(counts[:b]) + i for b in range(2) for i in {0, counts[b] // 2, counts[b] - 1}]
    mask = tree_masks(3, counts, empty=empty)
    for m in (None, mask):
        ref, A = definition(c, m)
        assert np.isnan(ref).any() and (m is None) == np.isnan(ref).all()
        same_but_where_nan(attend(c, m), ref, A, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 1, 16), (4, 2, 256)])
def test_decode_of_infinite_scores(hq, hkv, d, dtype):
    c = Case(63, [0, 40, -1, 5000], [1] * 4, hq, hkv, d, 16, dtype)
    c.k[..., 5] = INF
    ref, A = definition(c, decode=True)
    same_but_where_nan(gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale), ref, A, dtype)
    assert np.isnan(ref[[0, 1, 3]]).all() and not ref[2].any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hq,hkv,d,counts", [(8, 2, 128, [2, 3]), (8, 2, 128, [100, 40]), (8, 2, 64, [300, 40]), (4, 1, 256, [40, 2]), (4, 1, 16, [40, 2])])
def test_queries_of_a_row_that_is_not_in_use(hq, hkv, d, counts, dtype):
    # nothing writes them in a padded batch: they may be anything
    c = Case(64, [-1, 50], counts, hq, hkv, d, 16, dtype)
    c.q[:counts[0]] = NAN
    for mask in (None, tree_masks(4, counts)):
        o = attend(c, mask)
        assert not torch.any(o[:counts[0]].isnan()) and not torch.any(o[:counts[0]])
        c.q[:counts[0]] = 1.0
        assert torch.equal(attend(c, mask), o)
        c.q[:counts[0]] = NAN
    one = Case(65, [-1, 50], [1, 1], hq, hkv, d, 16, dtype)
    one.q[0] = NAN
    assert not torch.any(gb.gdn_kv_decode(one.q, *one.cache, scale=one.scale)[0])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hq,hkv,d,lens,counts", [(8, 2, 128, [50, 33], [3, 3]), (8, 2, 128, [300, 33], [40, 40]), (8, 2, 64, [500, 3], [130, 9]), (4, 1, 256, [90, 3], [70, 9]),
                                                  (8, 1, 128, [5000, 20], [2, 1]), (8, 1, 128, [5000, 20], [60, 1]), (4, 1, 256, [5000, 20], [60, 1])])
def test_tokens_that_see_a_key_of_nan_are_nan(hq, hkv, d, lens, counts, dtype):
    n = counts[0]
    c = Case(66, lens, counts, hq, hkv, d, 16, dtype)
    mask = tree_masks(5, counts)
    for m in (mask, None):
        clean = attend(c, m)
        for j in (0, n // 2, -lens[0], -(lens[0] // 2), -1):  # new tokens, then committed ones
            page, row = OA.slot(c.table.cpu().numpy(), 0, lens[0] + j, 16)
            kept = c.k[page, row].clone()
            c.k[page, row, :, 3] = NAN
            got = attend(c, m)
            c.k[page, row] = kept
            seen = np.ones(n, dtype=bool) if j < 0 else OA.bits(mask.cpu().numpy(), n)[:n, j] if m is not None else np.arange(n) >= j
            seen = torch.from_numpy(np.concatenate([seen, np.zeros(counts[1], dtype=bool)])).cuda()
            assert torch.all(got[seen].isnan()) and torch.equal(got[~seen], clean[~seen])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hq,hkv,d", [(64, 1, 64), (65, 1, 128), (128, 1, 128), (128, 2, 256), (129, 1, 64), (256, 2, 128)])
def test_many_query_heads_to_one(hq, hkv, d, dtype):
    counts, lens = [3, 1, 7], [200, 1100, 0]
    c = Case(67, lens, counts, hq, hkv, d, 16, dtype)
    for mask in (None, tree_masks(6, counts, empty=(1,))):
        close(attend(c, mask), *c.oracle(mask), dtype)
    one = Case(68, [200, 1100, 0, -1], [1] * 4, hq, hkv, d, 16, dtype)
    close(gb.gdn_kv_decode(one.q, *one.cache, scale=one.scale), *one.oracle(decode=True), dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size", [3e4, 3e5, 1e7])
@pytest.mark.parametrize("hq,hkv,d,lens,counts", [(8, 2, 128, [20, 300], [3, 4]), (8, 2, 128, [20, 300], [40, 3]), (4, 1, 64, [1000, 0], [300, 2]), (8, 1, 256, [500, 70], [30, 9]),
                                                  (8, 1, 128, [5000, 3], [60, 1])])
def test_scores_far_past_what_their_softmax_can_tell_apart(hq, hkv, d, lens, counts, size, dtype):
    # scores of 1e9 to 1e15, finite: the largest one has all the weight (their distances, 1e-3 of them and more here, are far more
    # than fp32 sums of d products are off, 2^-20 of their terms' sizes)
    c = Case(70, lens, counts, hq, hkv, d, 16, dtype)
    c.k *= size
    c.q *= size
    for mask in (None, tree_masks(7, counts)):
        ref, A = definition(c, mask)
        rows = sure_rows(c, mask)
        assert rows.mean() > 0.8
        o = attend(c, mask)
        assert torch.isfinite(o).all()
        close(torch.where(torch.from_numpy(rows)[..., None].cuda(), o, torch.zeros_like(o)), np.where(rows[..., None], ref, 0.0), np.where(rows[..., None], A, 0.0), dtype)


def sure_rows(c, mask):
    """[T, Hq]: whether a row's two largest scores differ by more than 2^-18 of the sum of their terms' sizes."""
    q, k = f64(c.q), np.nan_to_num(f64(c.k))
    table, off, group = c.table.cpu().numpy(), c.off.cpu().numpy(), c.q.shape[1] // c.k.shape[2]
    sure = np.ones(q.shape[:2], dtype=bool)
    bits = None if mask is None else OA.bits(mask.cpu().numpy(), max(c.counts))
    for b, n in enumerate(c.counts):
        at = [OA.slot(table, b, s, k.shape[1]) for s in range(c.lens_list[b] + n)]
        keys = np.stack([k[p, r] for p, r in at])
        for i in range(n):
            seen = np.concatenate([np.ones(c.lens_list[b], dtype=bool), np.arange(n) <= i if bits is None else bits[off[b] + i, :n]])
            for h in range(q.shape[1]):
                mine, row = keys[seen, h // group], q[off[b] + i, h]
                two = np.sort(mine @ row)[-2:]
                if len(two) == 2:
                    sure[off[b] + i, h] = two[1] - two[0] > 2.0 ** -18 * np.max(np.abs(mine) @ np.abs(row))
    return sure
