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


# cu_nodes of a batch, and the sequences of it that are good (inside the packed nodes, not decreasing, not beginning before an earlier entry)
MALFORMED = [
    ([0, 3, 2, 9], [0]),
    ([0, 5, 3, 9], [0]),
    ([0, 3, 7, 10], [0, 1]),
    ([1, 3, 7, 9], [1, 2]),
    ([0, -1, 7, 9], [2]),
    ([0, 20, 3, 7, 9], []),
    ([0, 4, 4, 2, 4, 9], [0, 1, 4]),
    ([0, 9, 0, 9, 0, 9, 0], [0]),
]


@pytest.mark.parametrize("cu,good", MALFORMED, ids=range(len(MALFORMED)))
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("ahead", [0, 300, 2500])  # good sequences ahead: later rounds of the lengths' check and of the packing
def test_malformed_lengths(kda, cu, good, draft, ahead):
    """Good sequences get what they get alone; the others accept nothing and have no token."""
    if ahead and cu[0]:
        pytest.skip("only the first sequence of all has to begin at 0")
    N, T = ahead + len(cu) - 1, ahead + 9
    c = _case([1] * T, 500, ref.F32, False, draft, seed=ahead + len(cu))
    chain = torch.randint(0, 500, (T,), generator=torch.Generator().manual_seed(3)).int()
    c.update(tokens=chain, us=c["us"][:N], cu=torch.tensor(list(range(ahead)) + [ahead + x for x in cu], dtype=torch.int32))
    c["ua"] *= 0.2  # (some tokens stand)
    out, status = _run(kda, c)
    assert status == kda.KDA_ERR_BAD_SEQLENS
    left = list(range(ahead)) + [ahead + n for n in good]
    spans = [(int(c["cu"][n]), int(c["cu"][n + 1])) for n in left]
    at = torch.cat([torch.arange(a, b) for a, b in spans] + [torch.zeros(0, dtype=torch.long)])
    part = dict(c, cu=ref.offsets([b - a for a, b in spans]), us=c["us"][left])
    for key in ("tokens", "target", "draft", "ua"):
        part[key] = c[key][at] if c[key] is not None else None
    want = ref.verify(part["tokens"], part["cu"], None, part["target"], part["draft"], part["ua"], part["us"])
    counts, tokens = np.zeros(N, dtype=np.int64), np.full(N, -1)
    counts[left], tokens[left] = np.diff(want[0]), want[2]
    rows = np.full(T, -1)
    rows[:want[0][-1]] = at.numpy()[want[1][:want[0][-1]]]
    assert out[0].tolist() == [0] + np.cumsum(counts).tolist()
    assert out[1].tolist() == rows.tolist() and out[2].tolist() == tokens.tolist()
