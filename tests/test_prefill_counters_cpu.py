"""The recurrent prompt kernel counts a prompt's tokens a tile past its end: with 2^31 - 1 of them that is more
than an int holds (heads of 16 with q, k and v in one array do fit the GPU)."""
import os
import re

from gated_delta_net_gb300 import build


def test_token_counters_hold_a_prompt_of_any_length_and_a_tile():
    text = open(os.path.join(build.CSRC, "prefill_simt.cu")).read()
    for name in ("n = inside", "t0 = 0", "t0) {"):
        kinds = re.findall(r"(\w+) %s" % re.escape(name), text)
        assert kinds and set(kinds) == {"unsigned"}, (name, kinds)
