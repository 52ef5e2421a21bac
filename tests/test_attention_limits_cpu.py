"""Sizes of gdn_attention.h at which places would leave 32 bits: refused before anything is launched."""
import ctypes

import pytest

from gated_delta_net_gb300 import binding as gb
from gated_delta_net_gb300 import build
from tests.test_attention_abi_cpu import APPEND, ATTEND, DECODE, UNSUPPORTED, _fill

WIDE = dict(d=256, page_stride=16 << 8, slot_stride=256, head_stride=256)


@pytest.fixture(scope="module")
def L():
    build.build()
    return gb.lib()


@pytest.mark.parametrize("heads", [1 << 23, (1 << 23) + 2, 1 << 28])
@pytest.mark.parametrize("fn,struct,sizes", [("gdn_kv_append", gb.KvAppendArgs, dict(APPEND, batch=1, total_tokens=1)),
                                             ("gdn_kv_attend", gb.KvAttendArgs, dict(ATTEND, batch=1, total_tokens=1, max_tokens=1)),
                                             ("gdn_kv_decode", gb.KvAttendArgs, dict(DECODE, batch=1, total_tokens=1))])
def test_rows_of_2_to_the_31_entries(L, fn, struct, sizes, heads):
    # (the pools' pointers are NULL, which is looked at later: nothing could be launched)
    null = dict(k_cache=None, v_cache=None, lens=None)
    for few in (2, heads):
        a = _fill(struct, sizes, **WIDE, **null, n_q_heads=heads, n_kv_heads=few)
        assert getattr(L, fn)(ctypes.byref(a), None) == UNSUPPORTED
        assert "2^31" in L.gdn_last_error().decode()
    if struct is gb.KvAppendArgs:  # keys and values only
        a = _fill(struct, sizes, **WIDE, **null, n_q_heads=0, n_kv_heads=heads, q=None)
        assert L.gdn_kv_append(ctypes.byref(a), None) == UNSUPPORTED
    else:
        assert L.gdn_kv_attend_workspace(ctypes.byref(_fill(struct, sizes, **WIDE, n_q_heads=heads, n_kv_heads=2)), fn == "gdn_kv_decode") == -1


def test_the_largest_row_is_taken_as_far_as_the_pointers(L):
    a = _fill(gb.KvAttendArgs, dict(DECODE, batch=1, total_tokens=1), **WIDE, n_q_heads=(1 << 23) - 1, n_kv_heads=1, lens=None)
    assert L.gdn_kv_decode(ctypes.byref(a), None) == gb.GDN_ERR_INVALID_ARG
