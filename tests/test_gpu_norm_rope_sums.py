"""The gradient of the norms' weights: every row counts, its error does not grow with the number of rows, and none is left unwritten.

A term is off by 40 half steps u = 2^-24 of fp32 (test_gpu_norm_rope.py).  A thread adds up at most 130 of them plainly, in whatever direction
their roundings go; a CTA's threads make 20 additions more, and joining those sums is exact to a few u: 200 u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from tests import _rollout_reference as roll
from tests import _spec_reference as ref
from tests._helpers import ensure_built

pytestmark = pytest.mark.gpu
U = roll.U


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


# few tokens of many heads, and many tokens of few: long sums of one thread (60 of 64 channels turned, or 126 of 128: rows through shared memory)
LONG = [(2, 65536, 0, 64, 64), (2, 40000, 20000, 64, 60), (300000, 4, 1, 64, 64), (250001, 2, 2, 64, 60), (3, 9000, 0, 1024, 1010)]


@pytest.mark.parametrize("T,Hq,Hk,d,rot", LONG)
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_long_sums_of_equal_rows(kda, T, Hq, Hk, d, rot, dtype):
    """Rows that are all alike, so that a plain sum's roundings all go one way."""
    gen = torch.Generator().manual_seed(T + d)
    freq, m = kda.rope_frequencies(rot)
    pos = torch.full((1,), 77, dtype=torch.int32)
    row, g = torch.randn(1, 1, d, generator=gen).to(dtype), torch.randn(1, 1, d, generator=gen).to(dtype)
    w = (1 + 0.3 * torch.randn(d, generator=gen)).to(dtype)
    _, dw, _, size = roll.norm_rope_bwd(row, w, g, pos.numpy(), freq.cpu().numpy(), 1e-6, False, m)
    heads = lambda x, H: x.cuda().expand(T, H, d).contiguous() if H else None  # noqa: E731
    wk = w.cuda() if Hk else None
    got = kda.kda_norm_rope_bwd(heads(row, Hq), heads(row, Hk), heads(g, Hq), heads(g, Hk), pos.cuda().expand(T).contiguous(), freq, w.cuda(), wk)
    for out, H in ((got[2], Hq), (got[3], Hk)):
        if H:
            off = np.abs(ref.np64(out) - T * H * dw) / (T * H * size)
            assert off.max() <= 200 * U, float(off.max() / U)


@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(2500, 12, 4, 64, 32), (2501, 7, 3, 128, 128), (1217, 5, 2, 128, 126), (4099, 1, 1, 256, 64), (70001, 2, 1, 64, 60)])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_every_token_counts(kda, T, Hq, Hk, d, rot, dtype):
    """One token alone has a gradient, the last one or one in between: dw is what that token alone gives."""
    gen = torch.Generator().manual_seed(T)
    x = [torch.randn(T, h, d, generator=gen).to(dtype) for h in (Hq, Hk)]
    pos = torch.randint(0, 5000, (T,), generator=gen, dtype=torch.int32)
    w = (1 + 0.3 * torch.randn(d, generator=gen)).to(dtype)
    freq, m = kda.rope_frequencies(rot)
    dev = [t.cuda() for t in x]
    for t in (T - 1, T - 2, T // 2 + 1, T // 3, 0):
        g = [torch.zeros(T, h, d, dtype=dtype) for h in (Hq, Hk)]
        for y in g:
            y[t] = torch.randn(y.shape[1], d, generator=gen).to(dtype)
        got = kda.kda_norm_rope_bwd(*dev, g[0].cuda(), g[1].cuda(), pos.cuda(), freq, w.cuda(), w.cuda())
        for i in range(2):
            dx, dw, _, size = roll.norm_rope_bwd(x[i][t:t + 1], w, g[i][t:t + 1], pos[t:t + 1].numpy(), freq.cpu().numpy(), 1e-6, False, m)
            assert np.all(np.abs(ref.np64(got[2 + i]) - dw) <= 200 * U * size)
            assert not bool(got[i][:t].any()) and not bool(got[i][t + 1:].any()) and bool(got[i][t].any())


def test_random_rows_by_the_norm_of_the_gradient(kda):
    """30,000 random rows: the terms' errors and the sums' have random signs, a few u of the gradient's norm together (1e-6 is 17 u); one row
    left out would be about 1 / sqrt(30,000) of it."""
    T, Hq, Hk, d = 2500, 12, 4, 64
    gen = torch.Generator().manual_seed(5)
    x, g = ([torch.randn(T, h, d, generator=gen) for h in (Hq, Hk)] for _ in "xg")
    pos = torch.randint(0, 5000, (T,), generator=gen, dtype=torch.int32)
    w = 1 + 0.3 * torch.randn(d, generator=gen)
    freq, m = kda.rope_frequencies(32)
    got = kda.kda_norm_rope_bwd(*(t.cuda() for t in (*x, *g)), pos.cuda(), freq, w.cuda(), w.cuda(), interleaved=True)
    for i in range(2):
        _, dw, _, _ = roll.norm_rope_bwd(x[i], w, g[i], pos.numpy(), freq.cpu().numpy(), 1e-6, True, m)
        assert np.linalg.norm(ref.np64(got[2 + i]) - dw) <= 1e-6 * np.linalg.norm(dw)


def test_outputs_for_an_absent_k_are_refused(kda):
    """Without k there is nothing to write into them: they would stay as they were."""
    q, pos = torch.randn(4, 2, 64, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    freq, _ = kda.rope_frequencies(64)
    held = torch.full((4, 2, 64), 7.0, device="cuda")
    with pytest.raises(ValueError):
        kda.kda_norm_rope(q, None, pos, freq, k_out=held)
    for bad in (dict(d_k=held), dict(d_k_weight=held[0, 0].contiguous())):
        with pytest.raises(ValueError):
            kda.kda_norm_rope_bwd(q, None, q, None, pos, freq, **bad)


@pytest.mark.parametrize("d,rot", [(64, 0), (64, 32), (128, 64), (128, 20), (128, 126), (136, 16), (256, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_channels_that_are_not_turned_know_nothing_of_one_another(kda, d, rot, interleaved, dtype):
    """An infinity among them: its head's other channels become zeros (its norm is infinite), and in the gradient its own weight's sum alone is no
    number or infinite."""
    gen = torch.Generator().manual_seed(d + rot)
    T, H = 6, 3
    x, g = (torch.randn(T, H, d, generator=gen).to(dtype) for _ in "xg")
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.rand(rot // 2, generator=gen, dtype=torch.float64).cuda()
    w = torch.ones(d, device="cuda")
    for at in range(rot, d, 5):
        y = x.clone()
        y[2, 1, at] = float("inf")
        out = kda.kda_norm_rope(y.cuda(), None, pos, freq, w, interleaved=interleaved)[0][2, 1]
        rest = torch.arange(d, device="cuda") != at
        assert bool((out[rest] == 0).all()) and bool(out[at].isnan())
        z = g.clone()
        z[2, 1, at] = float("inf")
        dw = kda.kda_norm_rope_bwd(x.cuda(), None, z.cuda(), None, pos, freq, w, interleaved=interleaved)[2]
        same = kda.kda_norm_rope_bwd(x.cuda(), None, g.cuda(), None, pos, freq, w, interleaved=interleaved)[2]
        assert torch.equal(dw[rest], same[rest]) and not bool(dw[at].isfinite())


@pytest.mark.parametrize("T,Hq,Hk,d", [(5, 3, 1, 64), (700, 4, 2, 128), (2, 40000, 2, 64), (3, 9000, 1, 136)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_gradient_stays_infinite(kda, T, Hq, Hk, d, sign):
    """One infinite entry of the output's gradient: that channel's sum is infinite, of its sign, and no other channel knows of it."""
    gen = torch.Generator().manual_seed(T)
    q, k = (torch.randn(T, h, d, generator=gen).abs() + 0.1 for h in (Hq, Hk))
    gq, gk = (torch.randn(T, h, d, generator=gen) for h in (Hq, Hk))
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda")
    w = torch.ones(d, device="cuda")
    call = lambda g: kda.kda_norm_rope_bwd(q.cuda(), k.cuda(), g.cuda(), gk.cuda(), pos, freq, w, w)  # noqa: E731
    plain, at = call(gq), (T - 1, Hq // 2, 21)
    gq[at] = sign * float("inf")
    got = call(gq)
    assert float(got[2][21]) == sign * float("inf")
    rest = torch.arange(d) != 21
    assert torch.equal(got[2][rest], plain[2][rest]) and torch.equal(got[3], plain[3])
    row = torch.zeros(T, Hq, dtype=torch.bool)
    row[at[:2]] = True
    assert bool(got[0][row].isnan().any()) and torch.equal(got[0][~row], plain[0][~row])
