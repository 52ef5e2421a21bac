"""Calls of the layer operators on two streams that are not ordered, with memory of the calls' own."""
import numpy as np
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from tests.test_gpu_layer import BF, offsets, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_net_gb300 import build
    build.build()
    gb.lib()


def test_segmented_prompts_on_two_streams_at_once():
    # two long prompts of few heads: both calls take a workspace of the same size, one right after the other
    T, hv = 4096, 2
    assert gb.gdn_prefill_workspace(1, 1, hv, 128, 128, T, T) > 0
    xs = [tokens(50 + i, T, 1, hv, 128, 128, BF, slow=True) for i in range(2)]
    off = offsets([T])
    refs = []
    for x in xs:
        refs.append(gb.gdn_prefill(*x, off, T))
        torch.cuda.synchronize()
    for kind in (lambda s: s, lambda s: s.cuda_stream):
        side = torch.cuda.Stream()
        for _ in range(5):
            here = [gb.gdn_prefill(*xs[0], off, T) for _ in range(3)]
            there = [gb.gdn_prefill(*xs[1], off, T, stream=kind(side)) for _ in range(3)]
            torch.cuda.synchronize()
            for got, ref in ((here, refs[0]), (there, refs[1])):
                for o, S in got:
                    assert torch.equal(o, ref[0]) and torch.equal(S, ref[1])


def test_results_of_another_stream_that_are_dropped_at_once():
    # what a call on the side stream returned goes back to the allocator while the call may still write it
    T, hv, d = 3000, 4, 128
    x = tokens(52, T, 2, hv, d, d, BF)
    w = torch.linspace(.5, 1.5, d).cuda()
    ref = gb.gdn_norm_gate(x[2], x[2], w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for _ in range(3):
            gb.gdn_norm_gate(x[2], x[2], w, stream=side)
        ones = torch.ones(T, hv, d, dtype=BF, device="cuda")
        got = gb.gdn_norm_gate(x[2], x[2], w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, ref) and np.all(ones.float().cpu().numpy() == 1.0)


def test_names_of_the_default_stream():
    x = tokens(53, 5, 1, 2, 64, 64, BF)
    w = torch.ones(64, device="cuda")
    ref = gb.gdn_norm_gate(x[2], x[2], w)
    torch.cuda.synchronize()
    for handle in (0, 1, 2):
        got = gb.gdn_norm_gate(x[2], x[2], w, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
