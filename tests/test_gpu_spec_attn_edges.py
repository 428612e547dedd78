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
@pytest.mark.parametrize("dtype,G", [(ref.BF16, 1), (ref.BF16, 8), (ref.F32, 2)])  # 8: trees of the tcgen05 kernel among them
@pytest.mark.parametrize("ahead", [0, 300])  # good sequences ahead: the plan's later rounds
def test_malformed_lengths(kda, cu, good, dtype, G, ahead):
    """Good sequences get what they get alone, every other row is left alone."""
    N, T, rng = ahead + len(cu) - 1, ahead + 9, np.random.default_rng(5)
    ctx = [int(x) for x in rng.integers(0, 130, N)]
    c = _case([1] * T, ctx + [0] * (T - N), G, 2, 64, 128, 16, dtype, False, seed=3)  # (sizes of T nodes, tables of N sequences)
    c.update(ctx=c["ctx"][:N], table=c["table"][:N], cu=torch.tensor(list(range(ahead)) + [ahead + x for x in cu], dtype=torch.int32))
    if ahead and cu[0]:
        pytest.skip("only the first sequence of all has to begin at 0")
    o, lse, status = _marked(kda, c)
    assert status == kda.KDA_ERR_BAD_SEQLENS
    want_o, want_lse = torch.full_like(o, 7), torch.full_like(lse, 7)
    left = [n for n in list(range(ahead)) + [ahead + n for n in good] if c["cu"][n] < c["cu"][n + 1]]
    spans = [slice(int(c["cu"][n]), int(c["cu"][n + 1])) for n in left]
    part = dict(c, ctx=c["ctx"][left], table=c["table"][left], cu=ref.offsets([s.stop - s.start for s in spans]))
    if left:
        for key in "qkv":
            part[key] = torch.cat([c[key][s] for s in spans])
        a, b, ok = _run(kda, part)
        assert ok == kda.KDA_OK
        at = torch.cat([torch.arange(s.start, s.stop) for s in spans]).cuda()
        want_o[at], want_lse[at] = a, b
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse)


def test_overlapping_trees_stay_inside_the_workspace(kda):
    """Four trees of 64 nodes over the same 64 packed nodes, each of several row tiles and parts: one counts, and nothing is written
    past the workspace."""
    ctx, cu = [4096] * 8, [0, 64] * 4 + [0]
    c = _case([64], [4096], 8, 4, 128, 128, 64, ref.BF16, True, seed=2)
    want = _run(kda, c)
    need = kda.kda_tree_attn_workspace_size(8, 64, 32, 4, 128, 64, 4096)
    whole = torch.full((need + (1 << 20),), 0xa5, dtype=torch.uint8, device="cuda")
    f = dict(c, ctx=torch.tensor(ctx, dtype=torch.int32), table=c["table"].expand(8, -1).contiguous(),
             cu=torch.tensor(cu, dtype=torch.int32))
    o, lse, status = _run(kda, f, workspace=whole[:need])
    assert status == kda.KDA_ERR_BAD_SEQLENS
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert bool((whole[need:] == 0xa5).all())


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("ctx", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 70])
def test_context_right_below_the_limit(kda, dtype, ctx):
    """One cache row read 2^31 - 1 times (a row stride of zero): equal scores, so o is the value and lse the score plus the
    logarithm of the number of keys.  A part left out would change that by 2e-3; 456 parts of exact counts are summed with rounding."""
    Hkv, d = 1, 64
    row = lambda x: torch.full((1, 1, Hkv, d), x, dtype=dtype, device="cuda").expand(1, ctx, Hkv, d)  # noqa: E731
    q, k, v = (torch.full((1, 1, d), x, dtype=dtype, device="cuda") for x in (0.5, 0.25, 2.0))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(kda.kda_tree_attn_workspace_size(1, 1, 1, Hkv, d, 1, ctx), dtype=torch.uint8, device="cuda")
    o, lse = kda.kda_tree_attn(q, k, v, row(0.25), row(2.0), ints(0).view(1, 1), ints(ctx), ints(0, 1), max_nodes=1, workspace=ws)
    assert kda.kda_device_status(ws) == kda.KDA_OK
    assert np.abs(ref.np64(lse) - (1.0 + np.log(ctx + 1.0))).max() <= 456 * 2.0 ** -24 + 22 * 2.0 ** -22
    assert np.abs(ref.np64(o) - 2.0).max() <= 2.0 * (912 * 2.0 ** -24 + ref.HALF_STEP[dtype])
