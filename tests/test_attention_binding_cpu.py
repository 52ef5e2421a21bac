"""Devices and streams of the attention calls' tensors, with stand-ins for the device: nothing is launched."""
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from tests import test_binding_memory_cpu as mem
from tests.test_binding_devices_cpu import _counted, _refuses_each
from tests.test_binding_memory_cpu import Stream, device  # noqa: F401

B, T, HQ, HKV, D, PAGES, PAGE = 2, 6, 4, 2, 16, 5, 8
I32 = dict(dtype=torch.int32)


class Library(mem.Library):
    def __getattr__(self, name):
        if name == "gdn_kv_attend_workspace":
            return lambda *args: 1024
        return super().__getattr__(name)


@pytest.fixture
def calls_to(device, monkeypatch):  # noqa: F811
    library = Library()
    monkeypatch.setattr(gb, "lib", lambda: library)
    return library, device[1]


def pools():
    return mem.dev(PAGES, PAGE, HKV, D), mem.dev(PAGES, PAGE, HKV, D), mem.dev(B, 2, **I32), mem.ints(3, 0)


def calls(stream=None):
    dev, ints = mem.dev, mem.ints
    return {
        "append": lambda: gb.gdn_kv_append(dev(T, HQ, D), dev(T, HKV, D), dev(T, HKV, D), *pools(), token_offsets=ints(0, 4, T), cos_sin=dev(9, D),
                                           stream=stream),
        "attend": lambda: gb.gdn_kv_attend(dev(T, HQ, D), *pools(), ints(0, 4, T), 4, anc_mask=dev(T, 1, **I32), stream=stream),
        "decode": lambda: gb.gdn_kv_decode(dev(B, HQ, D), *pools(), stream=stream),
        "commit": lambda: gb.gdn_kv_commit(*pools(), ints(0, 4, T), ints(0, 1, 1), ints(2), stream=stream),
    }


def calls_with_everything():
    dev, ints = mem.dev, mem.ints
    ws = lambda: dev(2048, dtype=torch.uint8)  # noqa: E731
    return {
        "append": lambda: gb.gdn_kv_append(dev(T, HQ, D), dev(T, HKV, D), dev(T, HKV, D), *pools(), token_offsets=ints(0, 4, T), depth=dev(T, **I32),
                                           cos_sin=dev(9, D), q_weight=dev(D), k_weight=dev(D), q_out=dev(T, HQ, D), dev_status=ints(0)),
        "attend": lambda: gb.gdn_kv_attend(dev(T, HQ, D), *pools(), ints(0, 4, T), 4, anc_mask=dev(T, 1, **I32), out=dev(T, HQ, D), workspace=ws(),
                                           dev_status=ints(0)),
        "decode": lambda: gb.gdn_kv_decode(dev(B, HQ, D), *pools(), out=dev(B, HQ, D), workspace=ws(), dev_status=ints(0)),
        "commit": lambda: gb.gdn_kv_commit(*pools(), ints(0, 4, T), ints(0, 1, 1), ints(2), new_lens=ints(0, 0), dev_status=ints(0)),
    }


NAMES = ["append", "attend", "commit", "decode"]


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_on_another_device(calls_to, monkeypatch, name):
    _refuses_each(calls_to, monkeypatch, calls_with_everything, name)


@pytest.mark.parametrize("name", NAMES)
def test_a_device_that_is_not_the_current_one(calls_to, monkeypatch, name):
    _counted(monkeypatch, "all")
    with pytest.raises(ValueError):
        calls_with_everything()[name]()
    assert calls_to[0].streams == []


@pytest.mark.parametrize("side", [Stream(9), 9], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream(calls_to, name, side):
    library, made = calls_to
    got = calls(side)[name]()
    assert library.streams == [9]
    assert made and [owner for _, owner in made] == [9] * len(made)
    assert got.data_ptr() in {t.data_ptr() for t, _ in made} and got.recorded == [7]


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_the_current_stream(calls_to, name):
    library, made = calls_to
    calls()[name]()
    assert library.streams == [7]
    assert made and all(owner == 7 and not hasattr(t, "recorded") for t, owner in made)
