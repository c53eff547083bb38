"""The order that early launches rely on, in the sources: a paged-cache kernel lets the next
one be set up only behind its own wait for the work before it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "qwen3_gated_attention_gb300", "csrc_seq")
KERNELS = ("paged_attn.cu", "paged_evict.cu", "paged_weights.cu", "prompt_rows.cu")


@pytest.mark.parametrize("name", KERNELS)
def test_the_next_launch_comes_behind_the_wait(name):
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    statements = [x.strip() for x in re.split(r"[;{}]", code)]
    early = [i for i, x in enumerate(statements) if x == "pdl_launch_dependents()"]
    assert early and all(statements[i - 1] == "pdl_wait()" for i in early)


def test_moves_follow_a_selection():
    code = open(os.path.join(CSRC, "paged_evict.cu")).read()
    launches = re.findall(r"launch_paged\((\w+)", code)
    assert launches == ["paged_select_kernel", "paged_close_kernel", "paged_move_kernel"]
