"""Draft verification: whole numbers, equal to the walk by its definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests import _spec_reference as ref
from tests._helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


def _case(lengths, V, dtype, tree, draft, seed, sharp=2.0, noise=1.0):
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    T = int(sum(lengths))
    logits = sharp * torch.randn(T, V, generator=gen)
    q = torch.softmax(logits + noise * torch.randn(T, V, generator=gen), -1)
    cu = ref.offsets(lengths)
    parent = ref.random_parents(lengths, rng)
    chain = torch.cat([torch.arange(m) - 1 for m in lengths]) if T else torch.zeros(0)
    up = parent if tree else chain
    first = torch.repeat_interleave(cu[:-1].long(), torch.tensor(lengths))
    tokens = torch.multinomial(q[first + up.long().clamp(min=0)], 1, generator=gen)[:, 0].int()
    return dict(tokens=tokens, cu=cu, parent=parent if tree else None, target=torch.softmax(logits, -1).to(dtype),
                draft=q.to(dtype) if draft else None, ua=torch.rand(T, generator=gen), us=torch.rand(len(lengths), generator=gen))


def _run(kda, c, **kw):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    ws = torch.full((kda.kda_draft_verify_workspace_size(len(c["cu"]) - 1),), 0xff, dtype=torch.uint8, device="cuda")
    out = kda.kda_draft_verify(d["tokens"], d["cu"], d["target"], d["ua"], d["us"], parent=d["parent"], draft_probs=d["draft"],
                               workspace=ws, **kw)
    return out, kda.kda_device_status(ws)


def _check(kda, c):
    out, status = _run(kda, c)
    assert status == kda.KDA_OK
    want = ref.verify(c["tokens"], c["cu"], c["parent"], c["target"], c["draft"], c["ua"], c["us"])
    for name, a, b in zip(("cu_accept", "rows", "next_token"), out, want):
        assert np.array_equal(a.cpu().numpy(), b), name
    return want


@pytest.mark.parametrize("lengths", [[1], [6], [4] * 9, [1, 0, 17, 2, 64, 33], [5] * 70], ids=range(5))
@pytest.mark.parametrize("V", [1, 3, 1000, 4097, 33333])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_against_reference(kda, lengths, V, tree, draft, dtype):
    if V == 33333 and len(lengths) == 70:
        pytest.skip("large")
    _check(kda, _case(lengths, V, dtype, tree, draft, seed=V + len(lengths)))


@pytest.mark.parametrize("V", [131072, 160001])
def test_large_flat_vocabulary(kda, V):
    """Nearly flat rows have a border every 1 / V: the sums must be far more exact than fp32."""
    want = _check(kda, _case([3] * 24, V, ref.F32, False, True, seed=V, sharp=0.1, noise=0.1))
    assert len(set(want[2].tolist())) > 12


def test_many_refusals(kda):
    """Wide trees whose drafts are mostly wrong: the residual shrinks child by child."""
    for seed in range(6):
        c = _case([40, 64, 25], 600, ref.F32, True, True, seed=seed, noise=4.0)
        c["parent"] = torch.cat([torch.where(torch.arange(m) == 0, -1, (torch.arange(m) - 1) // 12) for m in (40, 64, 25)]).int()
        c["ua"] = 0.7 + 0.3 * c["ua"]
        _check(kda, c)


def test_certain_decisions(kda):
    c = _case([5, 5], 100, ref.F32, False, True, seed=1)
    c["ua"].zero_()  # every drafted token has mass: all are accepted
    want = _check(kda, c)
    assert want[0].tolist() == [0, 5, 10]
    c["draft"] = None
    assert _check(kda, c)[0].tolist() == [0, 5, 10]
    c = _case([5, 5], 100, ref.F32, False, True, seed=1)
    c["target"].zero_()
    c["target"][:, 7] = 1.0  # a certain target: greedy verification
    c["tokens"][:] = 7
    c["tokens"][8] = 3
    c["draft"].fill_(0.01)
    want = _check(kda, c)
    assert want[0].tolist() == [0, 5, 8] and want[2].tolist() == [7, 7]
    # numbers at the ends of [0, 1)
    c = _case([3] * 4, 1000, ref.F32, False, True, seed=2)
    c["us"] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.0, 1 - 2.0 ** -24])
    _check(kda, c)


def test_residual_without_mass(kda):
    """p = q leaves nothing after a refusal (which only u = 1 brings): the draw falls back on p; no mass at all gives -1."""
    c = _case([2, 2, 1], 50, ref.F32, False, True, seed=3)
    c["draft"] = c["target"].clone()
    c["ua"][:] = 1.0
    c["target"][4] = 0.0
    out, status = _run(kda, c)
    assert status == kda.KDA_OK
    want = ref.verify(c["tokens"], c["cu"], None, c["target"], c["draft"], c["ua"], c["us"])
    assert out[0].tolist() == [0, 1, 2, 3] == want[0].tolist()
    assert out[2].tolist() == want[2].tolist() and out[2][2] == -1
    c["target"][4] = float("nan")
    assert _run(kda, c)[0][2][2] == -1


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("draft", [False, True])
def test_strides_and_alignment(kda, dtype, draft):
    """Rows at every alignment, target and draft at different ones; columns beyond V hold NaN."""
    c = _case([7, 3], 2050, dtype, True, draft, seed=4)
    want = ref.verify(c["tokens"], c["cu"], c["parent"], c["target"], c["draft"], c["ua"], c["us"])
    for pad, lead in ((0, 1), (1, 0), (3, 2), (6, 5), (8, 0)):
        f = dict(c)
        for key, off in (("target", lead), ("draft", 2 * lead + 1)):
            if c[key] is not None:
                buf = torch.full((10 * (2050 + pad) + off,), float("nan"), dtype=dtype, device="cuda")
                f[key] = buf[off:].view(10, 2050 + pad)[:, :2050]
                f[key].copy_(c[key])
        out, status = _run(kda, f)
        assert status == kda.KDA_OK
        for a, b in zip(out, want):
            assert np.array_equal(a.cpu().numpy(), b)


def test_device_errors_accept_nothing(kda):
    c = _case([3, 4, 2], 100, ref.F32, True, True, seed=5)
    want = ref.verify(c["tokens"], c["cu"], c["parent"], c["target"], c["draft"], c["ua"], c["us"])
    for key, at, value in (("tokens", 5, 100), ("tokens", 4, -1), ("parent", 5, 2), ("parent", 4, -1)):
        f = dict(c)
        f[key] = c[key].clone()
        f[key][at] = value
        out, status = _run(kda, f)
        assert status == kda.KDA_ERR_BAD_TREE
        first, last = want[0][1], want[0][3] - want[0][2]
        assert out[0].tolist() == [0, first, first, first + last]
        assert out[1].tolist() == want[1][:first].tolist() + [r for r in want[1].tolist() if r >= 7] + [-1] * (9 - first - last)
        assert out[2].tolist() == [want[2][0], -1, want[2][2]]
    for cu in ([0, 3, 2, 9], [0, 3, 7, 10], [1, 3, 7, 9], [0, 5, 3, 9]):
        out, status = _run(kda, dict(c, parent=None, cu=torch.tensor(cu, dtype=torch.int32)))
        assert status == kda.KDA_ERR_BAD_SEQLENS
        assert 0 <= int(out[0][-1]) <= 9
    big = _case([65], 20, ref.F32, False, False, seed=6)
    out, status = _run(kda, big)
    assert status == kda.KDA_ERR_BAD_SEQLENS and out[0].tolist() == [0, 0] and out[2].tolist() == [-1]
    assert _run(kda, c)[1] == kda.KDA_OK


def test_batch_invariance_graph_and_padding(kda):
    c = _case([4] * 150, 5000, ref.F32, False, True, seed=7)
    out, _ = _run(kda, c)
    for n in (0, 77, 149):
        s = slice(4 * n, 4 * n + 4)
        one = dict(tokens=c["tokens"][s], cu=ref.offsets([4]), parent=None, target=c["target"][s], draft=c["draft"][s],
                   ua=c["ua"][s], us=c["us"][n:n + 1])
        alone, _ = _run(kda, one)
        assert alone[2][0] == out[2][n] and alone[0][1] == out[0][n + 1] - out[0][n]
    # packed arrays may be longer than the last sequence
    pad = {k: (torch.cat([v, v[:3]]) if k not in ("cu", "us") and v is not None else v) for k, v in c.items()}
    padded, status = _run(kda, pad)
    assert status == kda.KDA_OK and torch.equal(padded[0], out[0]) and torch.equal(padded[1][:600], out[1])
    assert padded[1][600:].tolist() == [-1] * 3
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.kda_draft_verify(d["tokens"], d["cu"], d["target"], d["ua"], d["us"], draft_probs=d["draft"])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out))
    side = torch.cuda.Stream()
    got = kda.kda_draft_verify(d["tokens"], d["cu"], d["target"], d["ua"], d["us"], draft_probs=d["draft"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out))


def test_refusals(kda):
    c = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in _case([3], 10, ref.F32, True, True, seed=8).items()}
    for bad in (dict(tokens=c["tokens"].long()), dict(target=c["target"].T), dict(draft=c["draft"][:, :9]),
                dict(draft=c["draft"].bfloat16()), dict(ua=c["ua"].double()), dict(us=c["ua"]), dict(parent=c["parent"][:2])):
        a = dict(c, **bad)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_draft_verify(a["tokens"], a["cu"], a["target"], a["ua"], a["us"], parent=a["parent"], draft_probs=a["draft"])
    empty = kda.kda_draft_verify(c["tokens"][:0], c["cu"][:1] * 0, c["target"][:0], c["ua"][:0], c["us"][:0])
    assert empty[0].tolist() == [0] and empty[2].numel() == 0
