"""Append to the paged cache: exact copies, nothing else touched."""
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


def _case(new, ctx, Hkv, dk, dv, page, dtype, picked, seed=0):
    gen = torch.Generator().manual_seed(seed)
    total = int(sum(new))
    src = 2 * total + 1 if picked else total
    c = dict(cu=ref.offsets(new), ctx=torch.tensor(ctx, dtype=torch.int32))
    c["kp"], c["vp"], c["table"] = ref.paged(np.add(new, ctx), page, Hkv, dk, dv, dtype, seed, fill=5.0)
    c["k"], c["v"] = (torch.randn(src, Hkv, d, generator=gen).to(dtype) for d in (dk, dv))
    c["rows"] = torch.randperm(src, generator=gen)[:total].int() if picked else None
    return c


def _want(c, skip_seq=(), skip_row=()):
    kp, vp, page = c["kp"].clone(), c["vp"].clone(), c["kp"].shape[1]
    cu, ctx = c["cu"].tolist(), c["ctx"].tolist()
    new = list(ctx)
    for n in range(len(ctx)):
        if n in skip_seq:
            continue
        new[n] = ctx[n] + cu[n + 1] - cu[n]
        for j in range(cu[n], cu[n + 1]):
            if j in skip_row:
                continue
            at = ctx[n] + j - cu[n]
            r = j if c["rows"] is None else int(c["rows"][j])
            kp[int(c["table"][n, at // page]), at % page] = c["k"][r]
            vp[int(c["table"][n, at // page]), at % page] = c["v"][r]
    return kp, vp, new


def _run(kda, c, **kw):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    ws = torch.full((256,), 0xff, dtype=torch.uint8, device="cuda")
    kp, vp = d["kp"].clone(), d["vp"].clone()
    new = kda.kda_cache_append(d["k"], d["v"], kp, vp, d["table"], d["ctx"], d["cu"], rows=d["rows"], workspace=ws, **kw)
    return kp, vp, new, kda.kda_device_status(ws)


def _check(kda, c, status=0, **kw):
    kp, vp, new, st = _run(kda, c)
    want = _want(c, **kw)
    assert st == status
    assert torch.equal(kp.cpu(), want[0]) and torch.equal(vp.cpu(), want[1]) and new.tolist() == want[2]


@pytest.mark.parametrize("new,ctx,page", [([1], [0], 16), ([3, 0, 1, 5], [15, 7, 0, 60], 16), ([200, 1, 77], [0, 64, 33], 24),
                                          ([2] * 100, list(range(100)), 1), ([1000], [3], 100)])
@pytest.mark.parametrize("Hkv,dk,dv", [(1, 64, 64), (2, 128, 64), (8, 128, 128), (3, 64, 128)])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("picked", [False, True])
def test_exact(kda, new, ctx, page, Hkv, dk, dv, dtype, picked):
    _check(kda, _case(new, ctx, Hkv, dk, dv, page, dtype, picked, seed=len(new) + page))


def test_special_values_keep_their_bits(kda):
    c = _case([2], [3], 1, 64, 64, 16, ref.BF16, False)
    bits = torch.arange(-64, 64, dtype=torch.int16).view(2, 1, 64) * 255
    c["k"] = bits.view(ref.BF16)
    kp, _, _, _ = _run(kda, c)
    page = int(c["table"][0, 0])
    assert torch.equal(kp[page, 3:5].view(torch.int16).cpu(), bits)


def test_padding_strides_and_orders(kda):
    """rows beyond cu[N] (as verification leaves them) are not read; fused k | v; heads before rows in the pool."""
    c = _case([3, 2], [10, 20], 2, 128, 128, 16, ref.BF16, True, seed=3)
    want = _want(c)
    f = dict(c, rows=torch.cat([c["rows"], torch.full((7,), -1, dtype=torch.int32)]))
    kp, vp, new, st = _run(kda, f)
    assert st == kda.KDA_OK and torch.equal(kp.cpu(), want[0]) and torch.equal(vp.cpu(), want[1]) and new.tolist() == want[2]
    T = c["k"].shape[0]
    fused = torch.cat([c["k"].reshape(T, -1), c["v"].reshape(T, -1)], 1).cuda()
    pools = [c[x].transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in ("kp", "vp")]
    kda.kda_cache_append(fused[:, :256].view(T, 2, 128), fused[:, 256:].view(T, 2, 128), *pools, c["table"].cuda(), c["ctx"].cuda(),
                         c["cu"].cuda(), rows=c["rows"].cuda())
    assert torch.equal(pools[0].cpu(), want[0]) and torch.equal(pools[1].cpu(), want[1])


def test_device_errors(kda):
    good = _case([3, 4, 2], [10, 30, 5], 2, 128, 128, 16, ref.BF16, True, seed=4)
    c = dict(good, table=good["table"].clone())
    c["table"][1, 2] = -1  # positions 32, 33 of sequence 1: rows 5 and 6
    _check(kda, c, kda.KDA_ERR_BAD_PAGE, skip_row=(5, 6))
    c["table"][1, 2] = good["kp"].shape[0]
    _check(kda, c, kda.KDA_ERR_BAD_PAGE, skip_row=(5, 6))
    for value in (-1, good["k"].shape[0]):
        c = dict(good, rows=good["rows"].clone())
        c["rows"][4] = value
        _check(kda, c, kda.KDA_ERR_BAD_SLOT, skip_row=(4,))
    for ctx in (-1, good["table"].shape[1] * 16 - 3, 2 ** 31 - 2):  # does not fit its block table
        _check(kda, dict(good, ctx=torch.tensor([10, ctx, 5], dtype=torch.int32)), kda.KDA_ERR_BAD_PAGE, skip_seq=(1,))
    for cu, bad in (([0, 3, 2, 9], (1, 2)), ([0, 3, 7, 10], (2,)), ([1, 3, 7, 9], (0,))):
        kp, vp, new, st = _run(kda, dict(good, cu=torch.tensor(cu, dtype=torch.int32)))
        assert st == kda.KDA_ERR_BAD_SEQLENS
        assert torch.isfinite(kp.float()).all()
    _check(kda, good)


def test_stream_graph_and_refusals(kda):
    c = _case([3, 2], [10, 20], 2, 128, 128, 16, ref.BF16, True, seed=3)
    want = _want(c)
    d = {k: v.cuda() for k, v in c.items()}
    args = (d["k"], d["v"], d["kp"], d["vp"], d["table"], d["ctx"], d["cu"])
    graph = torch.cuda.CUDAGraph()
    before = d["kp"].clone(), d["vp"].clone()
    with torch.cuda.graph(graph):
        new = kda.kda_cache_append(*args, rows=d["rows"])
    d["kp"].copy_(before[0])
    d["vp"].copy_(before[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d["kp"].cpu(), want[0]) and torch.equal(d["vp"].cpu(), want[1]) and new.tolist() == want[2]
    side = torch.cuda.Stream()
    new = kda.kda_cache_append(*args, rows=d["rows"], stream=side)
    side.synchronize()
    assert new.tolist() == want[2]
    with pytest.raises(kda.KdaError):
        kda.kda_cache_append(*args, rows=d["rows"], new_len=d["ctx"])  # the lengths may not be their own result
    for i, bad in ((0, d["k"].float()), (1, d["v"][:1]), (2, d["kp"][:, :8]), (5, d["ctx"].long()), (6, d["cu"][:2])):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_cache_append(*args[:i], bad, *args[i + 1:], rows=d["rows"])
