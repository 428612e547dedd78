"""Rotary positions and their gradient against 64-bit arithmetic.

Bounds: one rounding of the result (half a step of its type) and, for the fp32 arithmetic, 8 roundings of the
magnitudes that meet in an element (sine or cosine to 2 units in the last place, its scaling, two products, one sum)."""
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


def _close(got, want, mag, dtype):
    bound = np.abs(want) * ref.HALF_STEP[dtype] + 8 * ref.HALF_STEP[ref.F32] * mag * (1 + ref.HALF_STEP[dtype])
    assert np.all(np.abs(ref.np64(got) - want) <= bound), float(np.max(np.abs(ref.np64(got) - want) - bound))


def _inputs(T, Hq, Hk, d, dtype, seed, max_pos=131072):
    gen = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(T, h, d, generator=gen).to(dtype) for h in (Hq, Hk))
    return q, k, torch.randint(-5, max_pos, (T,), generator=gen, dtype=torch.int32)


@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(1, 1, 1, 64, 64), (3, 32, 8, 128, 128), (5, 6, 2, 128, 64), (7, 3, 3, 64, 20),
                                           (2, 4, 1, 72, 2), (33, 2, 1, 256, 0), (9, 5, 5, 128, 126), (513, 8, 2, 128, 128),
                                           (2, 2, 1, 1024, 1024), (4, 2, 2, 1024, 1010)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_forward_and_gradient(kda, T, Hq, Hk, d, rot, interleaved, dtype):
    q, k, pos = _inputs(T, Hq, Hk, d, dtype, seed=T + d)
    w, m = kda.rope_frequencies(rot, scaling="yarn", factor=8.0)
    for call, backward in ((kda.kda_rope, False), (kda.kda_rope_bwd, True)):
        got = call(q.cuda(), k.cuda(), pos.cuda(), w, interleaved=interleaved, mscale=m)
        for x, y in zip((q, k), got):
            _close(y, *ref.rope(x, pos.numpy(), w.cpu().numpy(), interleaved, m, backward), dtype)
    assert torch.equal(got[0][..., rot:].cpu(), q[..., rot:])  # the rest is copied bit for bit


def test_far_positions_lose_nothing(kda):
    """Angles are reduced exactly: whole turns are added in integers."""
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    q, _, _ = _inputs(6, 2, 1, 128, ref.F32, seed=3)
    w, _ = kda.rope_frequencies(128)
    got, none = kda.kda_rope(q.cuda(), None, pos.cuda(), w)
    assert none is None
    # the angle of the table's fp64 frequency, in turns, with the product exact in rationals
    from fractions import Fraction
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563")
    frac = np.array([[float((Fraction(int(p)) * Fraction(float(f)) / two_pi) % 1) for f in w.cpu()] for p in pos])
    c, s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
    a, b = ref.np64(q)[..., :64], ref.np64(q)[..., 64:]
    mag = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    # (the table's 1 / 2 pi is rounded to 2^-53 relative: 2^31 positions of one radian are 2^-22 turns off at most)
    want = np.concatenate([a * c - b * s, a * s + b * c], -1)
    assert np.all(np.abs(ref.np64(got) - want) <= 8 * 2.0 ** -24 * mag + 2 * np.pi * 2.0 ** -22 * mag)
    near = slice(0, 4)
    assert np.all(np.abs(ref.np64(got) - want)[near] <= 9 * 2.0 ** -24 * mag[near])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_matches_differences(kda, interleaved):
    """The map is linear: a central difference of a weighted sum is its gradient up to the sums' rounding."""
    q, k, pos = _inputs(3, 2, 1, 64, ref.F32, seed=9)
    w, m = kda.rope_frequencies(32, scaling="yarn", factor=2.0)
    gq, gk = (torch.randn(x.shape, generator=torch.Generator().manual_seed(5)) for x in (q, k))
    dq, _ = kda.kda_rope_bwd(gq.cuda(), gk.cuda(), pos.cuda(), w, interleaved=interleaved, mscale=m)
    for t, h, i in [(0, 0, 0), (1, 1, 1), (2, 0, 17), (2, 1, 31), (0, 1, 40)]:
        step = torch.zeros_like(q)
        step[t, h, i] = 1.0  # exact in both directions up to the rounding of q + 1
        up, down = (kda.kda_rope((q + e * step).cuda(), k.cuda(), pos.cuda(), w, interleaved=interleaved, mscale=m)[0]
                    for e in (1, -1))
        diff = float(((up - down).double().cpu() * gq.double()).sum() / 2)
        assert abs(diff - float(dq[t, h, i])) <= 64 * 2.0 ** -24 * float(gq.abs()[t, h].max()) * 4


def test_strides_and_in_place(kda):
    T, Hq, Hk, d = 37, 8, 2, 128
    gen = torch.Generator().manual_seed(1)
    fused = torch.randn(T, (Hq + 2 * Hk) * d, generator=gen).to(ref.BF16).cuda()
    q, k = fused[:, :Hq * d].view(T, Hq, d), fused[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    w, _ = kda.rope_frequencies(d)
    want = kda.kda_rope(q.contiguous(), k.contiguous(), pos, w)
    got = kda.kda_rope(q, k, pos, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = fused[:, (Hq + Hk) * d:].clone()
    out = kda.kda_rope(q, k, pos, w, q_out=q, k_out=k)  # in place, inside the fused projection
    assert out[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(fused[:, (Hq + Hk) * d:], v)
    # rows that are not 16-byte aligned take the other path, with the same values
    odd = torch.empty(T * Hq * d + 1, dtype=ref.BF16, device="cuda")[1:].view(T, Hq, d)
    odd.copy_(got[0])
    back, _ = kda.kda_rope_bwd(odd, None, pos, w)
    even, _ = kda.kda_rope_bwd(got[0].contiguous(), None, pos, w)
    assert torch.equal(back, even)
    assert kda.kda_rope(q[:0], k[:0], pos[:0], w)[0].shape == (0, Hq, d)


def test_refusals(kda):
    q, k, pos = (x.cuda() for x in _inputs(4, 2, 1, 64, ref.BF16, seed=1))
    w, _ = kda.rope_frequencies(64)
    for bad in (dict(k=k.float()), dict(k=k[:3]), dict(pos=pos[:3]), dict(pos=pos.long()), dict(w=w.float()),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(q=q, k=k, pos=pos, w=w)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_rope(a["q"], a["k"], a["pos"], a["w"])
    with pytest.raises(kda.KdaError):
        kda.kda_rope(q, k, pos, kda.rope_frequencies(128)[0])  # rot > d
