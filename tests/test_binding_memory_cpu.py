"""Which stream the binding's own memory belongs to, with stand-ins for the device: nothing is launched.

A call with ``stream=`` has its results and its workspace written by that stream, so it takes them from memory
that torch keeps for that stream (a block of the current stream's may still be in use there, without an order
between the two), and records the current stream on what it returns.
"""
import contextlib
import ctypes

import pytest
import torch

from gated_delta_net_gb300 import binding as gb

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Stream:
    def __init__(self, cuda_stream, device=None):
        self.cuda_stream = cuda_stream


class Cuda(torch.Tensor):
    """CPU memory that says it is device memory."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = property(lambda self: True)
    device = property(lambda self: "cuda:0")

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream.cuda_stream]


class Library:
    """Takes every call and notes the stream it was given."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if name == "gdn_prefill_workspace":
                return 1024
            last = args[-1]
            self.streams.append(last.value or 0 if isinstance(last, ctypes.c_void_p) else last)
            return gb.GDN_OK
        return call


@pytest.fixture
def device(monkeypatch):
    """(library, made): ``made`` lists (tensor, stream that it was allocated for)."""
    library, made, current = Library(), [], [Stream(7)]
    real = torch.empty, torch.zeros

    def allocate(make):
        def f(*shape, dtype=None, device=None):
            t = make(*shape, dtype=dtype).as_subclass(Cuda)
            made.append((t, current[-1].cuda_stream))
            return t
        return f

    def empty_like(t, dtype=None):
        return torch.empty(tuple(t.shape), dtype=dtype or t.dtype)

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch, "empty", allocate(real[0]))
    monkeypatch.setattr(torch, "zeros", allocate(real[1]))
    monkeypatch.setattr(torch, "empty_like", empty_like)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: current[-1].cuda_stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(gb, "lib", lambda: library)
    return library, made


def dev(*shape, dtype=F32):
    return torch.ones(shape, dtype=dtype).as_subclass(Cuda)


def ints(*values):
    return torch.tensor(values, dtype=I32).as_subclass(Cuda)


T, HK, HV, D = 6, 1, 2, 16


def rule(n=T):
    return dev(n, HK, D), dev(n, HK, D), dev(n, HV, D), dev(n, HV), dev(n, HV)


LAYER = {
    "gdn_prefill": lambda s: gb.gdn_prefill(*rule(), ints(0, T), T, stream=s),
    "gdn_decode": lambda s: gb.gdn_decode(*rule(), dev(T, HV, D, D), stream=s),
    "gdn_qk_gates": lambda s: gb.gdn_qk_gates(*rule()[:2], dev(T, HV), dev(T, HV), dev(HV), dev(HV), stream=s),
    "gdn_norm_gate": lambda s: gb.gdn_norm_gate(dev(T, HV, D), dev(T, HV, D), dev(D), stream=s),
    "gdn_residual_norm": lambda s: gb.gdn_residual_norm(dev(T, 40), dev(T, 40), dev(40), stream=s),
}


NODES, PARENT = [0, T], [-1, 0, 1, 2, 3, 4]


def tree():
    return ints(*NODES), ints(*PARENT), dev(T, 1, dtype=I32), dev(T, dtype=I32)


PREV = dict(zip("k v g beta".split(), rule()[1:]), node_offsets=ints(*NODES), parent=ints(*PARENT),
            path_offsets=ints(0, 1), path_idx=ints(0))
TREE = {
    "build_desc": lambda s: gb.gdn_tree_build_desc(ints(*PARENT), ints(*NODES), T, stream=s),
    "states": lambda s: gb.gdn_tree_states(*rule()[1:], dev(1, HV, D, D), *tree()[:3], ints(0), ints(1), T, stream=s),
    "grow": lambda s: gb.gdn_tree_grow(ints(*NODES), dev(T, dtype=I32), dev(T, 2), 3, stream=s),
    "relabel": lambda s: gb.gdn_tree_relabel(ints(*PARENT), ints(*NODES), T, stream=s),
    "gather_rows": lambda s: gb.gdn_gather_rows(dev(T, 4), dev(T, dtype=I32), ints(*NODES), stream=s),
    "verify": lambda s: gb.gdn_tree_verify(*rule(), dev(1, HV, D, D), *tree(), T, stream=s),
    "verify_branches": lambda s: gb.gdn_tree_verify_branches(*rule(), dev(1, HV, D, D), *tree(), T, stream=s),
    "commit": lambda s: gb.gdn_tree_commit(*rule()[1:], dev(1, HV, D, D), *tree()[:2], ints(0, 1), ints(0), T, stream=s),
    "commit_nothing": lambda s: gb.gdn_tree_commit(*rule()[1:], dev(1, HV, D, D), *tree()[:2], ints(0, 0),
                                                   dev(0, dtype=I32), T, stream=s),
    "commit_verify": lambda s: gb.gdn_tree_commit_verify(PREV, dev(1, HV, D, D), T, 1, *rule(), *tree(), T, stream=s),
}
CALLS = {**LAYER, **TREE}


@pytest.mark.parametrize("side", [Stream(9), 9], ids=["stream", "handle"])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_of_a_call_on_another_stream(device, name, side):
    library, made = device
    got = CALLS[name](side)
    got = got if isinstance(got, tuple) else (got,)
    assert library.streams == [9]
    assert made and [owner for _, owner in made] == [9] * len(made)
    mine = {t.data_ptr() for t, _ in made}
    for t in got:
        assert t.data_ptr() in mine and t.recorded == [7]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_of_a_call_on_the_current_stream(device, name):
    library, made = device
    CALLS[name](None)
    assert library.streams == [7]
    assert made and all(owner == 7 and not hasattr(t, "recorded") for t, owner in made)


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_names_of_the_default_stream(device, handle):
    library, made = device
    gb.gdn_norm_gate(dev(T, HV, D), dev(T, HV, D), dev(D), stream=handle)
    assert library.streams == [handle] and [owner for _, owner in made] == [0]
