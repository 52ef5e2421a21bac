"""Host-side checks of gdn_layer.h that need no GPU: the exported entry points and the refusals
of bad arguments, which are made before anything is launched."""
import ctypes
import os
import re

import pytest

from gated_delta_net_gb300 import binding as gb
from gated_delta_net_gb300 import build

HEADER = os.path.join(build.INCLUDE, "gdn_layer.h")
INVALID, UNSUPPORTED = gb.GDN_ERR_INVALID_ARG, gb.GDN_ERR_UNSUPPORTED
FAKE = 0x1000  # never dereferenced: every case fails its checks, or is empty
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    build.build()
    return gb.lib()


def test_header_and_library_agree(L):
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"GDN_API\s+[\w\s\*]*?\b(gdn_\w+)\s*\(", text)))
    assert names == ["gdn_decode", "gdn_norm_gate", "gdn_prefill", "gdn_prefill_workspace", "gdn_qk_gates",
                     "gdn_residual_norm"]
    for name in names:
        assert hasattr(L, name), name


def _fill(struct, sizes, **kw):
    vals = {n: FAKE for n, t in struct._fields_ if t is ctypes.c_void_p}
    vals.update(workspace=None) if "workspace" in vals else None
    vals.update(sizes)
    vals.update(kw)
    return struct(**vals)


PREFILL = dict(batch=2, n_k_heads=1, n_v_heads=2, d_k=16, d_v=16, total_tokens=9, max_tokens=5, n_states=2, scale=1.0)
DECODE = dict(batch=2, n_k_heads=1, n_v_heads=2, d_k=16, d_v=16, n_states=2, scale=1.0)
GATES = dict(total_tokens=3, n_k_heads=1, n_v_heads=2, d_k=16, eps=1e-6)
NORM = dict(total_tokens=3, n_v_heads=2, d_v=16, eps=1e-6)
RESIDUAL = dict(total_tokens=3, width=40, scale=1.0, eps=1e-6)

RULE = [(dict(batch=-1), INVALID), (dict(n_k_heads=0), INVALID), (dict(n_k_heads=2, n_v_heads=3), INVALID),
        (dict(d_k=48), UNSUPPORTED), (dict(d_v=256), UNSUPPORTED), (dict(qkv_dtype=2), UNSUPPORTED),
        (dict(out_dtype=-1), UNSUPPORTED), (dict(n_states=-1), INVALID), (dict(scale=NAN), INVALID),
        (dict(q_stride=15), INVALID), (dict(k_stride=-16), INVALID), (dict(v_stride=31), INVALID),
        (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(beta=None), INVALID), (dict(o=None), INVALID)]
CASES = ([("gdn_prefill", gb.PrefillArgs, PREFILL, kw, code) for kw, code in RULE]
         + [("gdn_prefill", gb.PrefillArgs, PREFILL, kw, code) for kw, code in
            [(dict(total_tokens=-1), INVALID), (dict(max_tokens=-1), INVALID), (dict(token_offsets=None), INVALID),
             (dict(S_new=None), INVALID), (dict(S0=FAKE + 8), INVALID), (dict(S_new=FAKE + 4), INVALID)]]
         + [("gdn_decode", gb.DecodeArgs, DECODE, kw, code) for kw, code in
            RULE + [(dict(S=None), INVALID), (dict(S=FAKE + 4), INVALID)]]
         + [("gdn_qk_gates", gb.QkGatesArgs, GATES, kw, code) for kw, code in
            [(dict(total_tokens=-1), INVALID), (dict(n_k_heads=0), INVALID), (dict(n_v_heads=0), INVALID),
             (dict(d_k=24), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(eps=-1.0), INVALID),
             (dict(eps=NAN), INVALID), (dict(q_stride=8), INVALID), (dict(a_stride=1), INVALID),
             (dict(A_log=None), INVALID), (dict(g=None), INVALID), (dict(k_out=None), INVALID)]]
         + [("gdn_norm_gate", gb.NormGateArgs, NORM, kw, code) for kw, code in
            [(dict(total_tokens=-1), INVALID), (dict(n_v_heads=0), INVALID), (dict(d_v=24), UNSUPPORTED),
             (dict(act=2), UNSUPPORTED), (dict(weight_dtype=9), UNSUPPORTED), (dict(eps=-1.0), INVALID),
             (dict(z_stride=31), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID)]]
         + [("gdn_residual_norm", gb.ResidualNormArgs, RESIDUAL, kw, code) for kw, code in
            [(dict(total_tokens=-1), INVALID), (dict(width=0), INVALID), (dict(width=65537), UNSUPPORTED),
             (dict(dtype=3), UNSUPPORTED), (dict(scale=float("inf")), INVALID), (dict(eps=NAN), INVALID),
             (dict(x_stride=39), INVALID), (dict(y=None), INVALID), (dict(h=None), INVALID)]])


@pytest.mark.parametrize("fn,struct,sizes,kw,code", CASES)
def test_refusals(L, fn, struct, sizes, kw, code):
    a = _fill(struct, sizes, **kw)
    assert getattr(L, fn)(ctypes.byref(a), None) == code
    assert L.gdn_last_error().decode() != ""


@pytest.mark.parametrize("fn,struct,sizes", [("gdn_prefill", gb.PrefillArgs, dict(PREFILL, batch=0)),
                                             ("gdn_decode", gb.DecodeArgs, dict(DECODE, batch=0)),
                                             ("gdn_qk_gates", gb.QkGatesArgs, dict(GATES, total_tokens=0)),
                                             ("gdn_norm_gate", gb.NormGateArgs, dict(NORM, total_tokens=0)),
                                             ("gdn_residual_norm", gb.ResidualNormArgs, dict(RESIDUAL, total_tokens=0))])
def test_nothing_to_do_is_fine_and_null_args_are_not(L, fn, struct, sizes):
    a = struct(**sizes)
    assert getattr(L, fn)(ctypes.byref(a), None) == gb.GDN_OK
    assert getattr(L, fn)(None, None) == INVALID


def test_workspace_size_refuses_what_prefill_refuses(L):
    assert L.gdn_prefill_workspace(ctypes.byref(_fill(gb.PrefillArgs, PREFILL, d_k=48))) == -1
    assert L.gdn_prefill_workspace(ctypes.byref(_fill(gb.PrefillArgs, PREFILL))) >= 0
    with pytest.raises(gb.GdnError):
        gb.gdn_prefill_workspace(1, 2, 3, 16, 16, 4, 4)
