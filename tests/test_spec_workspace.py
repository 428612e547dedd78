"""Workspace of tree attention on the host: sizes that a batch can ask for, by type, and no more than that."""
import pytest
import torch

from tests._helpers import ensure_built


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("N,T,Hq,nodes,width,most", [
    (128, 512, 32, 4, 4096, 0.10), (128, 512, 32, 64, 4096, 0.10), (128, 512, 32, 64, 131072, 0.5),
    (256, 2048, 64, 8, 131072, 2.6), (128, 8192, 64, 64, 131072, 2.8)])
def test_serving_shapes(kda, N, T, Hq, nodes, width, most):
    """GiB of ordinary batches (8 KV heads of 128, bf16) whose block tables are as wide as the longest allowed context."""
    assert kda.kda_tree_attn_workspace_size(N, T, Hq, 8, 128, nodes, width, dtype=BF16) <= most * 2 ** 30


def test_sizes_by_type_and_bound(kda):
    size = kda.kda_tree_attn_workspace_size
    for args in ((4, 16, 16, 4, 128, 4, 9000), (3, 100, 8, 1, 64, 64, 700), (1, 1, 8, 8, 64, 1, 0), (5, 0, 8, 8, 64, 1, 100)):
        a, b = size(*args, dtype=BF16), size(*args, dtype=F32)
        assert size(*args) == max(a, b) and min(a, b) > 256
    # no tree has more nodes than the batch: a bound above that asks for nothing more
    assert size(1, 3, 32, 8, 128, 64, 9000, dtype=BF16) == size(1, 3, 32, 8, 128, 3, 9000, dtype=BF16)
    assert size(2, 8, 8, 2, 128, 4, 64, dtype=torch.float16) == 0 and size(2, 8, 9, 2, 128, 4, 64, dtype=BF16) == 0
