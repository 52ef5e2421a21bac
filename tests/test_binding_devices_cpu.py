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


@pytest.mark.parametrize("name", sorted(_layer()))
def test_a_tensor_on_another_device(device, monkeypatch, name):  # noqa: F811
    _refuses_each(device, monkeypatch, _layer, name)


@pytest.mark.parametrize("name", sorted(_layer()))
def test_a_device_that_is_not_the_current_one(device, monkeypatch, name):  # noqa: F811
    _counted(monkeypatch, "all")
    with pytest.raises(ValueError):
        _layer()[name]()
    assert device[0].streams == []
