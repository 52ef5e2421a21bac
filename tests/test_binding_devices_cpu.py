"""Tensors on other devices than the call's are refused before anything is launched (stand-ins for the device)."""
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from tests import test_binding_memory_cpu as mem
from tests.test_binding_memory_cpu import D, HK, HV, T, device  # noqa: F401


class Elsewhere(mem.Cuda):
    device = property(lambda self: "cuda:1")

    def get_device(self):
        return 1


def _layer():
    dev, ints, rule = mem.dev, mem.ints, mem.rule
    u8 = dict(dtype=torch.uint8)
    return {
        "gdn_prefill": lambda: gb.gdn_prefill(
            *rule(), ints(0, T), T, S0=dev(2, HV, D, D), slots=ints(1), fresh=ints(0), S_new=dev(2, HV, D, D),
            out=dev(T, HV, D), workspace=dev(2048, **u8), dev_status=ints(0)),
        "gdn_decode": lambda: gb.gdn_decode(*rule(), dev(T, HV, D, D), slots=ints(*range(T)), out=dev(T, HV, D), dev_status=ints(0)),
        "gdn_qk_gates": lambda: gb.gdn_qk_gates(dev(T, HK, D), dev(T, HK, D), dev(T, HV), dev(T, HV), dev(HV), dev(HV), q_out=dev(T, HK, D),
                                                k_out=dev(T, HK, D)),
        "gdn_norm_gate": lambda: gb.gdn_norm_gate(dev(T, HV, D), dev(T, HV, D), dev(D), out=dev(T, HV, D)),
        "gdn_residual_norm": lambda: gb.gdn_residual_norm(dev(T, 40), dev(T, 40), dev(40), post_weight=dev(40), h=dev(T, 40),
                                                          out=dev(T, 40)),
    }


def _tree():
    dev, ints, rule = mem.dev, mem.ints, mem.rule
    nodes, parents = [0, T], [-1, 0, 1, 2, 3, 4]
    i32 = dict(dtype=torch.int32)

    def tree():
        return ints(*nodes), ints(*parents), dev(T, 1, **i32), dev(T, **i32)

    def verify(fn):
        return lambda: fn(*rule(), dev(1, HV, D, D), *tree(), T, out=dev(T, HV, D), dev_status=ints(0))

    def fused():
        prev = dict(zip("k v g beta".split(), (dev(T, HK, D), dev(T, HV, D), dev(T, HV), dev(T, HV))), node_offsets=ints(*nodes),
                    parent=ints(*parents), path_offsets=ints(0, 1), path_idx=ints(0))
        return gb.gdn_tree_commit_verify(prev, dev(1, HV, D, D), T, 1, *rule(), *tree(), T, S_new=dev(1, HV, D, D),
                                         out=dev(T, HV, D), dev_status=ints(0))

    kv = lambda: (dev(T, HK, D), dev(T, HV, D), dev(T, HV), dev(T, HV))  # noqa: E731
    return {
        "build_desc": lambda: gb.gdn_tree_build_desc(ints(*parents), ints(*nodes), T, dev(T, 1, **i32), dev(T, **i32), dev_status=ints(0)),
        "states": lambda: gb.gdn_tree_states(*kv(), dev(1, HV, D, D), ints(*nodes), ints(*parents), dev(T, 1, **i32), ints(0),
                                             ints(1), T, out=dev(1, HV, D, D), dev_status=ints(0)),
        "grow": lambda: gb.gdn_tree_grow(ints(*nodes), dev(T, **i32), dev(T, 2), 3, dev_status=ints(0)),
        "relabel": lambda: gb.gdn_tree_relabel(ints(*parents), ints(*nodes), T, dev_status=ints(0)),
        "gather_rows": lambda: gb.gdn_gather_rows(dev(T, 4), dev(T, **i32), ints(*nodes), out=dev(T, 4), dev_status=ints(0)),
        "verify": verify(gb.gdn_tree_verify),
        "verify_branches": verify(gb.gdn_tree_verify_branches),
        "commit": lambda: gb.gdn_tree_commit(*kv(), dev(1, HV, D, D), ints(*nodes), ints(*parents), ints(0, 1), ints(0), T,
                                             out=dev(1, HV, D, D), dev_status=ints(0)),
        "commit_verify": fused,
    }


def _calls():
    return {**_layer(), **_tree()}


def _counted(monkeypatch, moved):
    """Make the tensors whose numbers are in ``moved`` (or all) elsewhere; returns the list of those made."""
    made = []

    def wrap(make):
        def f(*a, **kw):
            t = make(*a, **kw)
            if moved == "all" or len(made) in moved:
                t = t.as_subclass(Elsewhere)
            made.append(t)
            return t
        return f

    monkeypatch.setattr(mem, "dev", wrap(mem.dev))
    monkeypatch.setattr(mem, "ints", wrap(mem.ints))
    return made


def _refuses_each(device, monkeypatch, calls, name):
    library, _ = device
    with monkeypatch.context() as m:
        made = _counted(m, ())
        calls()[name]()
        n = len(made)
    assert len(library.streams) == 1
    for i in range(n):
        with monkeypatch.context() as m:
            _counted(m, (i,))
            with pytest.raises(ValueError):
                calls()[name]()
    assert len(library.streams) == 1


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_tensor_on_another_device(device, monkeypatch, name):  # noqa: F811
    _refuses_each(device, monkeypatch, _calls, name)


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_device_that_is_not_the_current_one(device, monkeypatch, name):  # noqa: F811
    _counted(monkeypatch, "all")
    with pytest.raises(ValueError):
        _calls()[name]()
    assert device[0].streams == []
