"""Edges of the attention operators (gdn_attention.h): what is not finite, and where it may not reach.

Cases and tolerances are those of test_gpu_attention; what has to be zero, NaN or unchanged is so exactly.
"""
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from oracle import attention as OA
from tests.test_gpu_attention import BF, F32, Case, tree_masks

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
