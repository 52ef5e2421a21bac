"""Kernels that are launched while the one before them in the stream may still run: a check of their source.

What the kernel before writes changes in their lifetime.  They wait for it before they touch global memory, and
read it with ordinary loads: a read-only load (__ldg) is defined for memory that stays as it is while the kernel
lives, and may be moved up past the wait.
"""
import glob
import os
import re

import pytest

from gated_delta_net_gb300 import build

READ_ONLY = re.compile(r"__ldg|__ldcs|__ldca|__ldcg|__ldlu|__ldcv|\.nc\b|__restrict__|prompt_length")


def _source(name):
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _early():
    return sorted(os.path.basename(p) for p in glob.glob(os.path.join(build.CSRC, "*.cu"))
                  if "launch_early(" in _source(os.path.basename(p)))


def test_there_are_some():
    assert _early() == ["decode.cu", "norms.cu"]


@pytest.mark.parametrize("name", ["decode.cu", "norms.cu"])
def test_they_wait_first_and_read_with_ordinary_loads(name):
    text = _source(name)
    assert READ_ONLY.findall(text) == []
    kernels = re.findall(r"__global__[^{;]*\)\s*\{\s*([^\n]*)", text)
    assert kernels and all(first.strip() == "after_previous();" for first in kernels)


@pytest.mark.parametrize("name", ["verify_tc.cu", "verify_wide.cu"])
def test_verification_after_a_commit_reads_its_state_with_coherent_loads(name):
    # launched while the commit that writes S0 runs; whatever holds S0's address in these files
    text = _source(name)
    names = {"S0"} | set(re.findall(r"(\w+) = (?:reinterpret_cast<[^>]*>\()?p\.S0\b", text))
    assert len(names) > 1
    for name in names:
        assert not re.search(r"__ld\w+\([^;]*\b%s\b" % name, text), name
