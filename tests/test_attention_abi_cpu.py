"""Host-side checks of gdn_attention.h that need no GPU: the exported entry points and the refusals of bad arguments,
which are made before anything is launched."""
import ctypes
import os
import re

import pytest

from gated_delta_net_gb300 import binding as gb
from gated_delta_net_gb300 import build

HEADER = os.path.join(build.INCLUDE, "gdn_attention.h")
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
    assert names == ["gdn_kv_append", "gdn_kv_attend", "gdn_kv_attend_workspace", "gdn_kv_commit", "gdn_kv_decode"]
    for name in names:
        assert hasattr(L, name), name


def test_structs_are_laid_out_as_the_header_says(tmp_path):
    import subprocess
    lines = []
    for struct, name in ((gb.KvAppendArgs, "gdn_kv_append_args"), (gb.KvAttendArgs, "gdn_kv_attend_args"), (gb.KvCommitArgs, "gdn_kv_commit_args")):
        lines.append(f"_Static_assert(sizeof({name}) == {ctypes.sizeof(struct)}, \"{name}\");")
        for field, _ in struct._fields_:
            at = {"k_cache": "cache.k", "v_cache": "cache.v"}.get(field, f"cache.{field}" if (field, _) in gb._CACHE else field)
            lines.append(f"_Static_assert(offsetof({name}, {at}) == {getattr(struct, field).offset}, \"{field}\");")
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include \"gdn_attention.h\"\n" + "\n".join(lines) + "\n")
    subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-I", build.INCLUDE, str(src)], check=True)


def _fill(struct, sizes, **kw):
    vals = {n: FAKE for n, t in struct._fields_ if t is ctypes.c_void_p}
    vals.update(sizes)
    vals.update(kw)
    return struct(**vals)


CACHE = dict(batch=2, n_pages=4, page_size=16, max_pages=3, n_kv_heads=2, d=64, page_stride=2048, slot_stride=128, head_stride=64)
APPEND = dict(CACHE, total_tokens=5, n_q_heads=4, rot_dim=32, n_positions=9, eps=1e-6)
ATTEND = dict(CACHE, max_pages=300, total_tokens=5, max_tokens=3, n_q_heads=4, mask_words=1, scale=1.0, workspace_bytes=1 << 40)
DECODE = dict(ATTEND, total_tokens=2)
COMMIT = dict(CACHE, total_path=3)

OF_CACHE = [(dict(batch=-1), INVALID), (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(max_pages=-1), INVALID),
            (dict(max_pages=1 << 30), UNSUPPORTED), (dict(n_kv_heads=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=512), UNSUPPORTED),
            (dict(dtype=2), UNSUPPORTED), (dict(page_stride=-1), INVALID), (dict(head_stride=-64), INVALID), (dict(k_cache=None), INVALID),
            (dict(v_cache=None), INVALID), (dict(page_table=None), INVALID), (dict(lens=None), INVALID)]
OF_ATTEND = [(dict(n_q_heads=3), INVALID), (dict(n_q_heads=0), INVALID), (dict(out_dtype=7), UNSUPPORTED), (dict(scale=NAN), INVALID),
             (dict(q_stride=255), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(o=FAKE + 8), INVALID),
             (dict(workspace=None), INVALID), (dict(workspace=FAKE + 128), INVALID), (dict(workspace_bytes=64), INVALID),
             (dict(total_tokens=-1), INVALID)]
CASES = ([("gdn_kv_append", gb.KvAppendArgs, APPEND, kw, code) for kw, code in OF_CACHE + [
            (dict(total_tokens=-1), INVALID), (dict(n_q_heads=3), INVALID), (dict(rot_dim=31), INVALID), (dict(rot_dim=66), INVALID),
            (dict(rot_dim=-2), INVALID), (dict(n_positions=-1), INVALID), (dict(weight_dtype=5), UNSUPPORTED), (dict(eps=NAN), INVALID),
            (dict(eps=-1.0), INVALID), (dict(q_stride=255), INVALID), (dict(k_stride=127), INVALID), (dict(v_stride=-128), INVALID),
            (dict(token_offsets=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID),
            (dict(cos_sin=None), INVALID)]]
         + [("gdn_kv_attend", gb.KvAttendArgs, ATTEND, kw, code) for kw, code in OF_CACHE + OF_ATTEND + [
            (dict(max_tokens=-1), INVALID), (dict(mask_words=0), INVALID), (dict(mask_words=1 << 21), UNSUPPORTED),
            (dict(token_offsets=None), INVALID), (dict(total_tokens=1 << 29), UNSUPPORTED)]]
         + [("gdn_kv_decode", gb.KvAttendArgs, DECODE, kw, code) for kw, code in OF_CACHE + OF_ATTEND + [(dict(total_tokens=3), INVALID)]]
         + [("gdn_kv_commit", gb.KvCommitArgs, COMMIT, kw, code) for kw, code in OF_CACHE + [
            (dict(total_path=-1), INVALID), (dict(node_offsets=None), INVALID), (dict(path_offsets=None), INVALID),
            (dict(path_idx=None), INVALID), (dict(new_lens=FAKE), INVALID)]])


@pytest.mark.parametrize("fn,struct,sizes,kw,code", CASES)
def test_refusals(L, fn, struct, sizes, kw, code):
    a = _fill(struct, sizes, **kw)
    assert getattr(L, fn)(ctypes.byref(a), None) == code
    assert L.gdn_last_error().decode() != ""


@pytest.mark.parametrize("fn,struct,sizes", [("gdn_kv_append", gb.KvAppendArgs, dict(APPEND, total_tokens=0, batch=0)),
                                             ("gdn_kv_attend", gb.KvAttendArgs, dict(ATTEND, batch=0)),
                                             ("gdn_kv_attend", gb.KvAttendArgs, dict(ATTEND, total_tokens=0)),
                                             ("gdn_kv_attend", gb.KvAttendArgs, dict(ATTEND, max_tokens=0)),
                                             ("gdn_kv_decode", gb.KvAttendArgs, dict(DECODE, batch=0, total_tokens=0)),
                                             ("gdn_kv_commit", gb.KvCommitArgs, dict(COMMIT, batch=0))])
def test_nothing_to_do_is_fine_and_null_args_are_not(L, fn, struct, sizes):
    a = struct(**sizes)
    assert getattr(L, fn)(ctypes.byref(a), None) == gb.GDN_OK
    assert getattr(L, fn)(None, None) == INVALID


def test_workspace_size_refuses_what_attend_refuses(L):
    need = lambda decode=0, **kw: L.gdn_kv_attend_workspace(ctypes.byref(_fill(gb.KvAttendArgs, DECODE if decode else ATTEND, **kw)), decode)  # noqa: E731
    assert need(d=48) == -1 and need(1, n_q_heads=3) == -1 and need(1, total_tokens=3) == -1
    assert need() > 0 and need(1) > 0 and need(total_tokens=0) == 0
    assert need() % 4 == 0
    assert need(1, max_pages=3) == 0  # no request long enough to be cut
    assert L.gdn_kv_attend_workspace(None, 0) == -1


KERNELS = ["kv_append.cu", "kv_commit.cu", "attend_simt.cu", "attend_mma.cu", "attend_tc.cu", "attn.cuh"]


@pytest.mark.parametrize("name", KERNELS)
def test_kernels_wait_for_the_one_before_them_and_read_with_ordinary_loads(name):
    # they may be launched while the kernel before them writes what they read
    text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
    assert not re.search(r"__ldg|__ldcs|__ldca|__ldcg|__ldlu|__ldcv|\.nc\b|__restrict__|prompt_length", text)
    kernels = re.findall(r"__global__[^{;]*\)\s*\{\s*([^\n]*)", text)
    assert kernels and all(first.strip() == "after_previous();" for first in kernels)
