"""Warps of the attention kernels stay together at their waits, also where one gives up: what follows is for whole warps (tcgen05 and
shuffles of all lanes).  A lane that left alone would leave the others waiting for it.  Read from the source: on a GPU only a wait that runs out
would show it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_linear_attention_chunk_gb300", "csrc")


def _body(text, head):
    at = text.index("{", re.search(head, text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]


@pytest.mark.parametrize("name, role", [(name, role) for name in ("kda_prefix_attn_tc.cu", "kda_tree_attn_tc.cu") for role in ("softmax", "fill")])
def test_no_lane_leaves_alone(name, role):
    with open(os.path.join(CSRC, name)) as f:
        body = _body(f.read(), r"__device__ \w+ " + role + r"\(")
    assert "wait_warp(" in body
    assert not re.search(r"(?<![\w])wait\(", body), "a wait whose lanes may part"
