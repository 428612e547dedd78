"""Tree attention over a paged cache against 64-bit arithmetic (bounds: _spec_reference.attn_bounds).

Cache rows beyond a sequence's context hold NaN and unused table entries point far outside the pool, so a row too
many shows in the result, or in the status."""
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


def _case(nodes, ctx, G, Hkv, dk, dv, page, dtype, tree, seed=0, sharp=1.0):
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    T = int(sum(nodes))
    c = dict(cu=ref.offsets(nodes), parent=ref.random_parents(nodes, rng) if tree else None,
             ctx=torch.tensor(ctx, dtype=torch.int32), scale=dk ** -0.5)
    c["kp"], c["vp"], c["table"] = ref.paged(ctx, page, Hkv, dk, dv, dtype, seed)
    c["q"] = (sharp * torch.randn(T, Hkv * G, dk, generator=gen)).to(dtype)
    c["k"], c["v"] = (torch.randn(T, Hkv, d, generator=gen).to(dtype) for d in (dk, dv))
    return c


def _dev(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _run(kda, c, **kw):
    d = _dev(c)
    ws = kw.pop("workspace", None)
    if ws is None:
        ws = torch.full((kda.kda_tree_attn_workspace_size(len(c["ctx"]), d["q"].shape[0], d["q"].shape[1], d["k"].shape[1],
                                                          d["v"].shape[2], kw.get("max_nodes", 64),
                                                          d["table"].shape[1] * d["kp"].shape[1]),), 0xff, dtype=torch.uint8, device="cuda")
    o, lse = kda.kda_tree_attn(d["q"], d["k"], d["v"], d["kp"], d["vp"], d["table"], d["ctx"], d["cu"], parent=d["parent"],
                               scale=c["scale"], workspace=ws, **kw)
    return o, lse, kda.kda_device_status(ws)


def _check(c, o, lse):
    dtype, dk = c["q"].dtype, c["q"].shape[2]
    want = ref.attn(c["q"], c["k"], c["v"], c["kp"], c["vp"], c["table"], c["ctx"], c["cu"], c["parent"], c["scale"])
    bo, bl = ref.attn_bounds(dtype, dk, int(c["ctx"].max()) + 64, *want)
    eo, el = np.abs(ref.np64(o) - want[0]), np.abs(ref.np64(lse) - want[1])
    assert np.all(eo <= bo), float((eo - bo).max())
    assert np.all(el <= bl), float((el - bl).max())


SHAPES = [
    # nodes, contexts, G, Hkv, dk, dv, page
    ([1], [0], 1, 1, 64, 64, 16),
    ([1, 1, 1], [1, 15, 16], 4, 2, 128, 128, 16),
    ([1], [700], 1, 3, 128, 128, 64),                        # one row, several parts
    ([4, 1, 0, 7], [63, 64, 5, 65], 4, 2, 128, 128, 24),     # an empty tree, pages that end inside a tile
    ([0, 0, 3], [9, 0, 0], 2, 1, 64, 128, 1),
    ([8, 3], [257, 1030], 4, 2, 128, 64, 100),
    ([16, 5, 13], [511, 0, 900], 3, 1, 128, 128, 8),         # 48 rows
    ([64, 33], [300, 1500], 1, 2, 64, 64, 32),
    ([64, 2, 40], [130, 2100, 77], 8, 1, 128, 128, 128),     # 512 rows: several row tiles
    ([17], [4099], 5, 2, 64, 128, 16),
    ([63, 64, 1, 31], [127, 128, 129, 640], 2, 1, 128, 64, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=range(len(SHAPES)))
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_against_reference(kda, shape, tree, dtype):
    c = _case(*shape, dtype, tree, seed=len(shape[0]) + shape[6])
    o, lse, status = _run(kda, c)
    assert status == kda.KDA_OK
    _check(c, o, lse)


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_sharp_scores_and_scales(kda, dtype):
    """Scores of some hundreds, both signs of the scale, and a scale of zero (plain means)."""
    for scale, sharp in ((128 ** -0.5, 12.0), (-0.05, 4.0), (0.0, 1.0)):
        c = _case([5, 2], [333, 70], 4, 2, 128, 128, 16, dtype, True, seed=4, sharp=sharp)
        c["scale"] = scale
        o, lse, status = _run(kda, c)
        assert status == kda.KDA_OK
        _check(c, o, lse)


def test_infinite_and_nan_keys_in_sight(kda):
    """What a row sees counts, as in the formula: a key of -inf scores takes no weight, NaN shows in that head alone."""
    c = _case([2], [100], 1, 2, 64, 64, 16, ref.F32, False, seed=2)
    c["q"] = c["q"].abs() + 0.1
    page, slot = int(c["table"][0, 3]), 5
    c["kp"][page, slot, 0] = -float("inf")
    d = dict(c)
    d["kp"] = c["kp"].clone()
    d["kp"][page, slot, 0] = -1e30  # the same weight: none
    o, lse, _ = _run(kda, c)
    _check(d, o, lse)
    c["kp"][page, slot, 0] = float("nan")
    o, lse, _ = _run(kda, c)
    assert bool(o[:, 0].isnan().all()) and bool(lse[:, 0].isnan().all()) and not bool(o[:, 1].isnan().any())


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_batch_invariance_and_repeatability(kda, dtype):
    nodes, ctx = [4, 1, 20, 64, 9], [900, 2000, 0, 555, 64]
    whole = _case(nodes, ctx, 4, 2, 128, 128, 16, dtype, True, seed=8)
    o, lse, _ = _run(kda, whole)
    o2, lse2, _ = _run(kda, whole)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    cu = whole["cu"].tolist()
    for n in range(len(nodes)):
        part = dict(whole, cu=ref.offsets([nodes[n]]), ctx=whole["ctx"][n:n + 1], table=whole["table"][n:n + 1])
        for key in ("q", "k", "v", "parent"):
            part[key] = whole[key][cu[n]:cu[n + 1]]
        a, b, _ = _run(kda, part, max_nodes=nodes[n])
        assert torch.equal(a, o[cu[n]:cu[n + 1]]) and torch.equal(b, lse[cu[n]:cu[n + 1]])


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("nodes", [2, 20])  # 16 and 160 query rows per KV head
def test_batch_size_changes_no_bits(kda, dtype, nodes):
    """A sequence of many parts alone, and among so many others that the parts are joined by the other kernels."""
    sizes, ctx = [nodes] + [64] * 9, [9000] + [3] * 9
    whole = _case(sizes, ctx, 8, 4, 128, 128, 64, dtype, True, seed=11)
    o, lse, _ = _run(kda, whole)
    alone = dict(whole, cu=ref.offsets([nodes]), ctx=whole["ctx"][:1], table=whole["table"][:1])
    for key in ("q", "k", "v", "parent"):
        alone[key] = whole[key][:nodes]
    a, b, _ = _run(kda, alone, max_nodes=nodes)
    assert torch.equal(a, o[:nodes]) and torch.equal(b, lse[:nodes])
    _check(alone, a, b)


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_infinite_value_in_sight(kda, dtype):
    c = _case([3], [100], 2, 4, 64, 64, 16, dtype, False, seed=2)
    page, slot = int(c["table"][0, 3]), 5
    c["vp"][page, slot, 1, 7] = float("inf")
    o, _, _ = _run(kda, c)
    assert bool(torch.isposinf(o[:, 2:4, 7]).all())
    o[:, 2:4, 7] = 0
    assert bool(torch.isfinite(o).all())


def test_padded_nodes_are_left_alone(kda):
    c = _case([3, 4], [70, 40], 4, 2, 128, 128, 16, ref.BF16, True, seed=7)
    want = _run(kda, c)
    padded = dict(c)
    for key in ("q", "k", "v", "parent"):
        padded[key] = torch.cat([c[key], c[key][:1].expand(3, *c[key].shape[1:])])
    o, lse, status = _marked(kda, padded)
    assert status == kda.KDA_OK and torch.equal(o[:7], want[0]) and torch.equal(lse[:7], want[1])
    assert bool((o[7:] == 7).all()) and bool((lse[7:] == 7).all())


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_strides_and_axis_orders(kda, dtype):
    """q, k, v inside one fused projection; heads before rows in the pools; K and V interleaved in one pool."""
    c = _case([6, 3], [200, 90], 4, 2, 128, 128, 16, dtype, True, seed=5)
    o, lse, _ = _run(kda, c)
    T = c["q"].shape[0]
    fused = torch.cat([c[x].reshape(T, -1) for x in "qkv"], 1).cuda()
    f = dict(c)
    f["q"], f["k"], f["v"] = fused[:, :1024].view(T, 8, 128), fused[:, 1024:1280].view(T, 2, 128), fused[:, 1280:].view(T, 2, 128)
    pool = torch.stack([c["kp"], c["vp"]], 1).permute(0, 1, 3, 2, 4).contiguous().cuda()  # [pages, 2, Hkv, page, d]
    f["kp"], f["vp"] = pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2)
    table = torch.full((2, c["table"].shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = c["table"].cuda()
    f["table"] = table[:, :c["table"].shape[1]]
    o2, lse2, status = _run(kda, f)
    assert status == kda.KDA_OK and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_offsets_past_32_bits(kda):
    """A pool of more than 2^32 bytes and 2^31 elements, addressed at both ends."""
    page, Hkv, d = 16, 2, 128
    stride = 2 ** 31 // 64 + 4096  # elements per page
    pool = torch.empty(66 * stride, dtype=ref.BF16, device="cuda")
    pages = pool.as_strided((66, page, Hkv, d), (stride, Hkv * d, d, 1))
    c = _case([3], [100], 4, Hkv, d, d, page, ref.BF16, True, seed=6)
    f = dict(c)
    far = torch.tensor([[65, 0, 64, 1, 63, 2, 62]], dtype=torch.int32)
    for key, at in (("kp", 0), ("vp", page * Hkv * d)):
        view = pool[at:].as_strided(pages.shape, pages.stride()) if at else pages
        view[far[0].long().cuda()] = c[key][c["table"][0].long()].cuda()
        f[key] = view
    f["table"] = far
    o, lse, status = _run(kda, f)
    assert status == kda.KDA_OK
    want = _run(kda, c)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def _marked(kda, c, **kw):
    """A run whose outputs hold 7 where nothing was written."""
    T, Hq, dv = c["q"].shape[0], c["q"].shape[1], c["v"].shape[2]
    o = torch.full((T, Hq, dv), 7.0, dtype=c["q"].dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    return _run(kda, c, o=o, lse=lse, **kw)


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("ctx1", [40, 1400])  # one part and several
def test_device_errors_write_nothing(kda, dtype, ctx1):
    nodes, ctx = [3, 4, 2], [70, ctx1, 33]
    good = _case(nodes, ctx, 4, 2, 128, 128, 16, dtype, True, seed=7)
    want = _run(kda, good)
    bad = {}
    bad[kda.KDA_ERR_BAD_PAGE] = [dict(good, table=good["table"].clone()), dict(good, table=good["table"].clone()),
                                 dict(good, ctx=torch.tensor([70, -1, 33], dtype=torch.int32)),
                                 dict(good, ctx=torch.tensor([70, 1 << 20, 33], dtype=torch.int32))]
    bad[kda.KDA_ERR_BAD_PAGE][0]["table"][1, 1] = -1
    bad[kda.KDA_ERR_BAD_PAGE][1]["table"][1, ctx1 // 16] = good["kp"].shape[0]
    bad[kda.KDA_ERR_BAD_TREE] = [dict(good, parent=good["parent"].clone()) for _ in range(2)]
    bad[kda.KDA_ERR_BAD_TREE][0]["parent"][5] = 2   # node 2 of sequence 1: not before itself
    bad[kda.KDA_ERR_BAD_TREE][1]["parent"][6] = -1
    for code, cases in bad.items():
        for c in cases:
            o, lse, status = _marked(kda, c)
            assert status == code
            assert bool((o[3:7] == 7).all()) and bool((lse[3:7] == 7).all())
            for a, b in ((o, want[0]), (lse, want[1])):
                assert torch.equal(a[:3], b[:3]) and torch.equal(a[7:], b[7:])
    # the next call starts with a clean status
    assert _run(kda, good)[2] == kda.KDA_OK


def test_bad_lengths(kda):
    good = _case([3, 4, 2], [70, 40, 33], 4, 2, 128, 128, 16, ref.BF16, False, seed=7)
    want = _run(kda, good)
    for cu, written in (([0, 3, 2, 9], [0, 1, 2]), ([0, 3, 7, 10], [0, 1, 2, 3, 4, 5, 6]), ([1, 3, 7, 9], [3, 4, 5, 6, 7, 8]),
                        ([0, -1, 7, 9], [7, 8])):
        o, lse, status = _marked(kda, dict(good, cu=torch.tensor(cu, dtype=torch.int32)))
        assert status == kda.KDA_ERR_BAD_SEQLENS
        assert torch.equal(o[written], want[0][written]) or cu[2] == 2
    o, _, status = _marked(kda, good, max_nodes=3)  # a tree larger than the caller said
    assert status == kda.KDA_ERR_BAD_SEQLENS and bool((o[3:7] == 7).all()) and torch.equal(o[:3], want[0][:3])


def test_streams_graph_and_no_lse(kda):
    c = _case([4, 9], [800, 90], 4, 2, 128, 128, 16, ref.BF16, True, seed=3)
    d = _dev(c)
    want, want_lse, _ = _run(kda, c)
    args = (d["q"], d["k"], d["v"], d["kp"], d["vp"], d["table"], d["ctx"], d["cu"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, lse = kda.kda_tree_attn(*args, parent=d["parent"], stream=side)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    o, none = kda.kda_tree_attn(*args, parent=d["parent"], return_lse=False)
    assert none is None and torch.equal(o, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = kda.kda_tree_attn(*args, parent=d["parent"])
    d["q"].mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    c["q"] = -c["q"]
    want = _run(kda, c)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_refusals(kda):
    c = _dev(_case([2, 2], [20, 30], 4, 2, 128, 128, 16, ref.BF16, True, seed=3))
    names = ("q", "k", "v", "kp", "vp", "table", "ctx", "cu")
    for bad in (dict(q=c["q"].float()), dict(k=c["k"][:, :1]), dict(v=c["v"][:3]), dict(kp=c["kp"][:, :8]), dict(kp=c["kp"].float()),
                dict(table=c["table"].long()), dict(ctx=c["ctx"][:1]), dict(cu=c["cu"][:2]), dict(parent=c["parent"][:3]),
                dict(kp=c["kp"].transpose(2, 3))):
        a = dict(c, **bad)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_tree_attn(*(a[x] for x in names), parent=a["parent"])
    with pytest.raises(kda.KdaError):
        kda.kda_tree_attn(*(c[x] for x in names), parent=c["parent"], max_nodes=65)
    with pytest.raises(kda.KdaError):
        kda.kda_tree_attn(*(c[x] for x in names), parent=c["parent"], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
