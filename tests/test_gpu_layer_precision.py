"""How far the chunked prompts are from exact, norm-wise for each head, beside the bounds of what they round.

States: an operand of the state's chain is a pair of bf16, off by at most 2^-18 of itself.  On the way to the
state stand four in a row (A, T, the operands W and S or T' and V, U'), at most 2^-16 together; they are not
aligned, and with unit keys that have nothing in common they average out to about 2^-18, so that 1e-5 holds with
a margin of two.  Gates, and what stands between two tokens, are good to fp32's 2^-24 times a few.

Outputs: bf16, so 2^-9 of themselves, and their products' operands S, U and Y once more each: with the terms'
own sizes at most 4 x 2^-9.
"""
import numpy as np
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from oracle import layer as OL
from tests.test_gpu_layer import BF, f64, offsets, pool, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_net_gb300 import build
    build.build()
    gb.lib()


def far(got, ref, axes):
    """The largest distance of a head's (or a row's) values from exact, relative to their norm."""
    got = f64(got)
    assert np.all(np.isfinite(got))
    return np.max(np.sqrt(np.sum((got - ref) ** 2, axis=axes) / np.sum(ref ** 2, axis=axes)))


@pytest.mark.parametrize("forgotten,decay", [(0, 0.0), (1, -np.inf), (4, -np.inf), (8, -90.0), (12, -np.inf), (13, -48.0)])
@pytest.mark.parametrize("before", [0, 64])
def test_prefill_slow_tokens_after_strong_decays(forgotten, decay, before):
    # tokens that forget (nearly) everything inside a block of 16, then slow ones whose keys have much in common
    T, hk, hv, d = before + 32, 2, 4, 128
    q, k, v, g, beta = tokens(60 + forgotten, T, hk, hv, d, d, BF, slow=True)
    k = torch.nn.functional.normalize(0.7 * k[:1].float() + 0.714 * k.float(), dim=-1).to(BF)
    g[before + 17:before + 17 + forgotten] = decay
    S0 = pool(61, 1, hv, d, d)
    o, S = gb.gdn_prefill(q, k, v, g, beta, offsets([T]), T, S0=S0)
    ro, rS = OL.prefill(*map(f64, (q, k, v, g, beta)), [0, T], S0=f64(S0))
    assert far(S, rS, (2, 3)) <= 2.0 ** -16
    assert far(o, ro, (0, 2)) <= 2.0 ** -7


@pytest.mark.parametrize("lengths", [[40], [130], [64, 300, 1000], [3000]], ids=str)
def test_prefill_states_and_outputs(lengths):
    hk, hv, d = 2, 4, 128
    x = tokens(62, sum(lengths), hk, hv, d, d, BF, slow=True)
    off = offsets(lengths)
    S0 = pool(63, len(lengths), hv, d, d)
    o, S = gb.gdn_prefill(*x, off, max(lengths), S0=S0, scale=d ** -0.5)
    ro, rS = OL.prefill(*map(f64, x), off.cpu().numpy(), S0=f64(S0), scale=d ** -0.5)
    assert far(S, rS, (2, 3)) <= 1e-5
    assert far(o, ro, (0, 2)) <= 2.0 ** -7
    assert far(o, ro, 2) <= 2.0 ** -5  # each row of its own, small ones too: a row's terms may cancel to a quarter


@pytest.mark.parametrize("lengths", [[64], [300, 1000], [3000]], ids=str)
def test_prefill_outputs_are_rounded_to_bf16_once(lengths):
    # rounding to bf16 is 2^-9 / sqrt(3) of a value's leading bit, 1.66e-3 norm-wise over mantissas of 1 to 2.  The
    # products' operands have 2^-12 of theirs (tf32) or less: two times 2^-12 / sqrt(3), of terms that are up to twice
    # the sum, leave it below 2^-9
    hk, hv, d = 2, 4, 128
    x = tokens(64, sum(lengths), hk, hv, d, d, BF, slow=True)
    off = offsets(lengths)
    S0 = pool(65, len(lengths), hv, d, d)
    o, _ = gb.gdn_prefill(*x, off, max(lengths), S0=S0, scale=d ** -0.5)
    ro, _ = OL.prefill(*map(f64, x), off.cpu().numpy(), S0=f64(S0), scale=d ** -0.5)
    assert far(o, ro, (0, 2)) <= 2.0 ** -9
