"""Single tokens and small drafts in bf16 lose no more than their outputs' own rounding to bf16.

Probabilities are two bf16 numbers as the operand beside the values: the first is off by 2^-8 of one, the second by 2^-8 of
that, 2^-16 together.  With A = sum_s p_s |v_s|, scores and sums add 2^-15 A (test_gpu_attention), and the outputs' own
rounding 2^-8 of them where they are bf16: 2^-8 |o| + (2^-16 + 2^-15) A.
"""
import numpy as np
import pytest

from gated_delta_net_gb300 import binding as gb
from tests.test_gpu_attention import BF, F32, Case, f64, tree_masks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_net_gb300 import build
    build.build()
    gb.lib()


def near(got, ref, A):
    own = 2.0 ** -8 * 1.01 if got.dtype == BF else 0.0
    over = np.abs(f64(got) - ref) - (own * np.abs(ref) + (2.0 ** -16 + 2.0 ** -15) * A + 1e-30)
    assert float(over.max()) <= 0, np.argwhere(over > 0)[:8].tolist()


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d,page,lens", [(8, 2, 128, 16, [300, 0, 77]), (4, 1, 16, 16, [500, 3]), (24, 1, 256, 64, [1000, 9]), (3, 3, 32, 5, [200]), (8, 1, 64, 16, [9000, 40]),
                                                (8, 2, 128, 16, [4000, -1, 1])])
def test_decode(hq, hkv, d, page, lens, out_dtype):
    c = Case(80 + d, lens, [1] * len(lens), hq, hkv, d, page, BF)
    near(gb.gdn_kv_decode(c.q, *c.cache, scale=c.scale, out_dtype=out_dtype), *c.oracle(decode=True))


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,d,lens,counts", [(8, 2, 128, [300, 20], [4, 2]), (4, 1, 256, [2000, 0], [3, 4]), (2, 1, 64, [700, 5], [8, 6]), (4, 4, 16, [90, 5], [16, 2])])
def test_small_drafts(hq, hkv, d, lens, counts, out_dtype):
    c = Case(90 + d, lens, counts, hq, hkv, d, 16, BF)
    for mask in (None, tree_masks(20, counts)):
        near(gb.gdn_kv_attend(c.q, *c.cache, c.off, max(counts), anc_mask=mask, scale=c.scale, out_dtype=out_dtype), *c.oracle(mask))
