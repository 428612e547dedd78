"""Append to the paged cache where it can go wrong: malformed lengths, large batches.  Exact: nothing else is touched."""
import pytest
import torch

from tests import _spec_reference as ref
from tests._helpers import ensure_built
from tests.test_gpu_spec_append import _case, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


# cu of a batch, and the sequences of it that are bad (outside the rows, decreasing, or beginning before an earlier entry)
MALFORMED = [
    ([0, 3, 2, 9], (1, 2)),
    ([0, 5, 3, 9], (1, 2)),
    ([0, 3, 7, 10], (2,)),
    ([1, 3, 7, 9], (0,)),
    ([0, -1, 7, 9], (0, 1)),
    ([0, 20, 3, 7, 9], (0, 1, 2, 3)),
    ([0, 4, 4, 2, 4, 9], (2, 3)),
    ([0, 9, 0, 9, 0, 9, 0], (1, 2, 3, 4, 5)),
]


@pytest.mark.parametrize("cu,bad", MALFORMED, ids=range(len(MALFORMED)))
@pytest.mark.parametrize("Hkv,dk,dv,dtype", [(1, 64, 64, ref.BF16), (3, 64, 128, ref.F32), (16, 128, 128, ref.BF16)])
@pytest.mark.parametrize("picked", [False, True])
@pytest.mark.parametrize("ahead", [0, 300])
def test_malformed_lengths(kda, cu, bad, Hkv, dk, dv, dtype, picked, ahead):
    """A bad sequence keeps its length and writes nothing; the others are appended whole."""
    if ahead and cu[0]:
        pytest.skip("only the first sequence of all has to begin at 0")
    N = ahead + len(cu) - 1
    c = _case([9] * N, [(5 * n) % 23 for n in range(N)], Hkv, dk, dv, 16, dtype, picked, seed=4)  # (room for 9 rows in each)
    c["cu"] = torch.tensor(list(range(ahead)) + [ahead + x for x in cu], dtype=torch.int32)
    rows = ahead + 9
    if picked:
        c["rows"] = c["rows"][:rows]
    else:
        c["k"], c["v"] = c["k"][:rows], c["v"][:rows]
    _check(kda, c, kda.KDA_ERR_BAD_SEQLENS, skip_seq=tuple(ahead + n for n in bad))


def test_large_batches(kda):
    """More sequences than the lengths' check takes in one round, empty ones among them; several lengths per thread."""
    for N in (3000, 5000):
        _check(kda, _case([(0, 1, 3, 2)[i % 4] for i in range(N)], [(7 * n) % 40 for n in range(N)], 1, 64, 64, 8, ref.BF16, True, seed=N))
