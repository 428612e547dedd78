"""Tree attention where it can go wrong: ragged tiles, malformed lengths, masked infinities, far contexts, the tcgen05 kernel's
special cases.  Against 64-bit arithmetic (bounds: _spec_reference.attn_bounds)."""
import numpy as np
import pytest
import torch

from tests import _spec_reference as ref
from tests._helpers import ensure_built
from tests.test_gpu_spec_attn import _case, _check, _marked, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("nodes,G", [(1, 1), (5, 4), (20, 2)])
def test_rows_that_are_not_there(kda, dtype, dk, dv, nodes, G):
    """Tiles of which nearly every row is absent, in the first page of a pool that begins its allocation."""
    for ctx in (0, 1, 65):
        c = _case([nodes], [ctx], G, 1, dk, dv, 128, dtype, False, seed=ctx + nodes)
        if ctx:
            at = int(c["table"][0, 0])
            for key in ("kp", "vp"):
                c[key] = c[key][[at] + [i for i in range(c[key].shape[0]) if i != at]]
            c["table"][0, 0] = 0
        o, lse, status = _run(kda, c)
        assert status == kda.KDA_OK
        _check(c, o, lse)
