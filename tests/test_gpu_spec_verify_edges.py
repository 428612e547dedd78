"""Draft verification where it can go wrong: large batches, empty trees, malformed lengths, rows of several steps per segment."""
import numpy as np
import pytest
import torch

from tests import _spec_reference as ref
from tests._helpers import ensure_built
from tests.test_gpu_spec_verify import _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


@pytest.mark.parametrize("N", [225, 320, 700])  # more than a packing round, than two CTAs each, than are resident
@pytest.mark.parametrize("draft", [False, True])
def test_large_batches(kda, N, draft):
    """Empty trees end at once, the others after one or more passes: whichever is last packs them all."""
    lengths = [(0, 1, 3, 2)[i % 4] for i in range(N)]
    _check(kda, _case(lengths, 777, ref.F32, True, draft, seed=N))


def test_empty_trees_only(kda):
    c = _case([0] * 260, 50, ref.F32, False, True, seed=1)
    out, status = _run(kda, c)
    assert status == kda.KDA_OK
    assert out[0].tolist() == [0] * 261 and out[1].numel() == 0 and out[2].tolist() == [-1] * 260


@pytest.mark.parametrize("dtype,draft", [(ref.BF16, True), (ref.BF16, False), (ref.F32, False)])
def test_several_steps_per_segment(kda, dtype, draft):
    """Rows of more than 131,072 entries, refused tokens in later steps of their segments."""
    V = 300001
    c = _case([4, 6], V, dtype, True, draft, seed=9, sharp=0.5, noise=3.0)
    c["ua"] = 0.5 + 0.5 * c["ua"]
    _check(kda, c)
