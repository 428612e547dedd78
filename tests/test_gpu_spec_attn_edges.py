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


ODD = [  # nodes, contexts, G, Hkv, dk, dv: the register kernels' row groups, four heads per CTA (fp32), one and several row tiles, parts
    ([6], [0], 1, 1, 64, 64),
    ([5, 9, 1], [70, 1400, 3], 2, 4, 64, 128),
    ([13, 4], [900, 33], 2, 3, 128, 64),
    ([40, 7], [200, 2100], 1, 2, 128, 128),
    ([64, 11], [1300, 5], 8, 1, 128, 128),
    ([33], [5000], 8, 2, 64, 64),
]


@pytest.mark.parametrize("shape", ODD, ids=range(len(ODD)))
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_values_that_a_row_does_not_see(kda, shape, dtype):
    """Infinities and NaN in a drafted node's key and value: rows that do not see the node are what they are without them, rows that
    do have the infinity, or NaN, in that column (a key of NaN makes all of the row NaN)."""
    c = _case(*shape, 16, dtype, True, seed=len(shape[0]))
    nodes, _, G, Hkv, _, dv = shape
    cu = c["cu"].tolist()
    want_o, want_lse, status = _run(kda, c)
    assert status == kda.KDA_OK
    _check(c, want_o, want_lse)
    f = dict(c, k=c["k"].clone(), v=c["v"].clone())
    want_o, want_lse = want_o.cpu(), want_lse.cpu()
    n = int(np.argmax(nodes))
    sees = ref.ancestors([-1] + c["parent"][cu[n] + 1:cu[n + 1]].tolist())
    marks = [(nodes[n] - 1, 0, 3, float("inf")), (nodes[n] - 2, Hkv - 1, dv - 1, -float("inf")), (1, Hkv - 1, 0, float("nan")),
             (nodes[n] // 2, 0, 9, float("inf")), (2, 0, 9, -float("inf"))]
    for node, head, column, x in marks:
        f["v"][cu[n] + node, head, column] = x
    lost = nodes[n] - 1
    f["k"][cu[n] + lost, Hkv - 1] = float("nan")
    for i in range(nodes[n]):
        for head in range(Hkv):
            for column in range(dv):
                xs = [x for node, h, col, x in marks if h == head and col == column and sees[i, node]]
                if xs:
                    want_o[cu[n] + i, head * G:(head + 1) * G, column] = sum(xs)  # (both infinities: NaN)
            if head == Hkv - 1 and sees[i, lost]:
                want_o[cu[n] + i, head * G:(head + 1) * G] = float("nan")
                want_lse[cu[n] + i, head * G:(head + 1) * G] = float("nan")
    o, lse, status = _run(kda, f)
    assert status == kda.KDA_OK
    assert torch.equal(torch.nan_to_num(o.cpu(), nan=77.0, posinf=88.0, neginf=99.0),
                       torch.nan_to_num(want_o, nan=77.0, posinf=88.0, neginf=99.0))
    assert torch.equal(torch.nan_to_num(lse.cpu(), nan=77.0), torch.nan_to_num(want_lse, nan=77.0))


@pytest.mark.parametrize("dtype,nodes,G", [(ref.BF16, 4, 2), (ref.BF16, 40, 4), (ref.F32, 7, 2)])
def test_a_drafted_branch_changes_nothing_before_it(kda, dtype, nodes, G):
    """A chain's last node is all NaN: the nodes before it, and the other sequences, keep their bits."""
    c = _case([3, nodes, 2], [100, 300, 0], G, 4, 128, 128, 16, dtype, False, seed=6)
    want_o, want_lse, _ = _run(kda, c)
    last = 3 + nodes - 1
    f = dict(c, **{key: c[key].clone() for key in "qkv"})
    for key in "qkv":
        f[key][last] = float("nan")
    o, lse, status = _run(kda, f)
    assert status == kda.KDA_OK
    keep = [i for i in range(nodes + 5) if i != last]
    assert torch.equal(o[keep], want_o[keep]) and torch.equal(lse[keep], want_lse[keep])
    assert bool(o[last].isnan().all()) and bool(lse[last].isnan().all())


def _sizes(rng, N, most):
    return [int(rng.integers(1, most + 1)) if rng.random() < 0.5 else int(rng.choice([1, most])) for _ in range(N)]


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("N,most,G,Hkv,longest", [(1, 1, 1, 1, 9000), (9, 4, 4, 8, 9000), (5, 64, 8, 4, 20000), (40, 9, 8, 1, 3000), (6, 33, 5, 3, 9000)])
def test_partial_results_stay_inside_the_workspace(kda, dtype, N, most, G, Hkv, longest):
    """Batches of every mixture of tree sizes over contexts as long as their block tables allow, in a workspace of exactly the size
    that is asked for, with a marked region behind it."""
    rng = np.random.default_rng(N)
    nodes = _sizes(rng, N, most)
    c = _case(nodes, [longest if rng.random() < 0.8 else int(rng.integers(0, longest)) for _ in nodes], G, Hkv, 64, 64, 128, dtype, True, seed=N)
    width = c["table"].shape[1] * 128
    need = kda.kda_tree_attn_workspace_size(N, sum(nodes), G * Hkv, Hkv, 64, most, width, dtype=dtype)
    assert need <= kda.kda_tree_attn_workspace_size(N, sum(nodes), G * Hkv, Hkv, 64, most, width)
    whole = torch.full((need + (1 << 20),), 0xa5, dtype=torch.uint8, device="cuda")
    o, lse, status = _run(kda, c, workspace=whole[:need], max_nodes=most)
    assert status == kda.KDA_OK and bool((whole[need:] == 0xa5).all())
    _check(c, o, lse)


# ---- the tcgen05 kernel's special cases (bf16, more than 32 rows per KV head), beside sequences of the register kernels ----------

WIDE = dict(nodes=[3, 9, 2, 33], G=16, Hkv=2)  # 48, 144, 32 and 528 rows: a tile alone, a pair, the register kernel, pairs and one over


def _wide(ctx, dk, dv, page=16, tree=True, seed=0, sharp=1.0):
    return _case(WIDE["nodes"], ctx, WIDE["G"], WIDE["Hkv"], dk, dv, page, ref.BF16, tree, seed=seed, sharp=sharp)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128)])
@pytest.mark.parametrize("scale,sharp", [(None, 12.0), (-0.05, 4.0), (0.0, 1.0)])
def test_wide_sharp_scores_and_scales(kda, dk, dv, scale, sharp):
    c = _wide([333, 70, 1500, 2900], dk, dv, seed=4, sharp=sharp)
    c["scale"] = dk ** -0.5 if scale is None else scale
    o, lse, status = _run(kda, c)
    assert status == kda.KDA_OK
    _check(c, o, lse)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_wide_maximum_that_keeps_rising(kda, sign):
    """Scores that grow along the context by hundreds, so that the reference is left behind tile after tile; and that fall."""
    c = _wide([1000, 2000, 300, 700], 128, 128, page=64, seed=8)
    c["q"] = (c["q"].abs() + 0.5).to(ref.BF16)
    for n, length in enumerate(c["ctx"].tolist()):
        at = torch.arange(length)
        ramp = sign * torch.linspace(-3, 3, length)[:, None, None]
        page, slot = c["table"][n].long()[at // 64], at % 64
        c["kp"][page, slot] = (0.1 * c["kp"][page, slot].float() + ramp).to(ref.BF16)
    o, lse, status = _run(kda, c)
    assert status == kda.KDA_OK
    _check(c, o, lse)


@pytest.mark.parametrize("ctx1", [40, 1400, 6000])  # one part and several
def test_wide_device_errors_write_nothing(kda, ctx1):
    good = _wide([70, ctx1, 33, 500], 128, 128, seed=7)
    want = _run(kda, good)
    assert want[2] == kda.KDA_OK
    for code, key, at, value in ((kda.KDA_ERR_BAD_PAGE, "table", (1, 1), -1), (kda.KDA_ERR_BAD_PAGE, "table", (1, (ctx1 - 1) // 16), good["kp"].shape[0]),
                                 (kda.KDA_ERR_BAD_PAGE, "ctx", 1, -1), (kda.KDA_ERR_BAD_PAGE, "ctx", 1, 1 << 20),
                                 (kda.KDA_ERR_BAD_TREE, "parent", 5, 2), (kda.KDA_ERR_BAD_TREE, "parent", 11, -1)):
        f = dict(good)
        f[key] = good[key].clone()
        f[key][at] = value
        o, lse, status = _marked(kda, f)
        assert status == code
        assert bool((o[3:12] == 7).all()) and bool((lse[3:12] == 7).all())
        for a, b in ((o, want[0]), (lse, want[1])):
            assert torch.equal(a[:3], b[:3]) and torch.equal(a[12:], b[12:])
    assert _run(kda, good)[2] == kda.KDA_OK


def test_wide_strides_and_axis_orders(kda):
    """q, k, v inside one fused projection; heads before rows in the pools; K and V in one pool; a wider block table."""
    c = _wide([200, 90, 1000, 10], 128, 128, seed=5)
    o, lse, _ = _run(kda, c)
    T, Hq, Hkv = c["q"].shape[0], 32, 2
    fused = torch.cat([c[x].reshape(T, -1) for x in "qkv"], 1).cuda()
    f = dict(c)
    f["q"] = fused[:, :Hq * 128].view(T, Hq, 128)
    f["k"], f["v"] = (fused[:, (Hq + i * Hkv) * 128:(Hq + (i + 1) * Hkv) * 128].view(T, Hkv, 128) for i in range(2))
    pool = torch.stack([c["kp"], c["vp"]], 1).permute(0, 1, 3, 2, 4).contiguous().cuda()  # [pages, 2, Hkv, page, d]
    f["kp"], f["vp"] = pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2)
    table = torch.full((4, c["table"].shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = c["table"].cuda()
    f["table"] = table[:, :c["table"].shape[1]]
    o2, lse2, status = _run(kda, f)
    assert status == kda.KDA_OK and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_wide_offsets_past_32_bits(kda):
    page, Hkv, d = 16, 2, 128
    stride = 2 ** 31 // 64 + 4096  # elements per page
    pool = torch.empty(66 * stride, dtype=ref.BF16, device="cuda")
    pages = pool.as_strided((66, page, Hkv, d), (stride, Hkv * d, d, 1))
    c = _case([3], [100], 16, Hkv, d, d, page, ref.BF16, True, seed=6)
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


@pytest.mark.parametrize("ctx", [100, 3000])
def test_wide_infinities_and_nan_in_sight(kda, ctx):
    """What a row sees counts: an infinite value in its column, a key of -inf scores not at all, a key of NaN in that head."""
    c = _case([3], [ctx], 16, 2, 64, 64, 16, ref.BF16, False, seed=2)
    c["q"] = c["q"].abs() + 0.1
    page, slot = int(c["table"][0, 3]), 5
    f = dict(c, vp=c["vp"].clone(), kp=c["kp"].clone())
    f["vp"][page, slot, 1, 7] = float("inf")
    o, _, _ = _run(kda, f)
    assert bool(torch.isposinf(o[:, 16:, 7]).all())
    o[:, 16:, 7] = 0
    assert bool(torch.isfinite(o).all())
    f = dict(c, kp=c["kp"].clone())
    f["kp"][page, slot, 0] = -float("inf")
    o, lse, _ = _run(kda, f)
    f["kp"][page, slot, 0] = -1e30  # the same weight: none
    _check(f, o, lse)
    f["kp"][page, slot, 0] = float("nan")
    o, lse, _ = _run(kda, f)
    assert bool(o[:, :16].isnan().all()) and bool(lse[:, :16].isnan().all()) and not bool(o[:, 16:].isnan().any())


@pytest.mark.parametrize("dtype,G", [(ref.BF16, 1), (ref.BF16, 12), (ref.F32, 2)])
def test_large_batches(kda, dtype, G):
    """More sequences than the plan takes in one round, empty ones among them, trees of every kernel."""
    rng = np.random.default_rng(3)
    N = 700
    nodes = [int(x) for x in rng.choice([0, 1, 2, 3, 9], N)]
    ctx = [int(x) for x in rng.integers(0, 300, N)]
    c = _case(nodes, ctx, G, 1, 64, 64, 16, dtype, True, seed=9)
    o, lse, status = _run(kda, c)
    assert status == kda.KDA_OK
    _check(c, o, lse)


def test_default_bound_on_nodes_changes_no_bits(kda):
    for nodes, G in (([1], 4), ([1, 1, 1], 8), ([4, 1, 3], 4), ([5, 2], 8)):
        c = _case(nodes, [900, 40, 7][:len(nodes)], G, 2, 128, 128, 16, ref.BF16, True, seed=len(nodes))
        a, b = _run(kda, c), _run(kda, c, max_nodes=max(nodes))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
