"""Probabilities of unlikely and masked tokens, and what the integer masses leave of long tails.

A probability is off by the roundings of its exponential (exp2f: two units in the last place, 4 half steps of fp32; what goes into it: a
quarter), of the total and its inverse (2) and of their product (1), with 2e-10 and half a unit per token for the total (a quarter): 8 half
steps 2^-24 of it.  Where fp32 has no such number, by its smallest step; then comes the rounding to its type."""
import numpy as np
import pytest
import torch

from tests import _rollout_reference as roll
from tests import _spec_reference as ref
from tests._helpers import ensure_built

pytestmark = pytest.mark.gpu
SMALLEST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133}


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


def _probs(kda, logits, probs_dtype, **filters):
    """The call's distributions, checked against the definition."""
    N = logits.shape[0]
    u = torch.full((N,), 0.375)
    out = torch.full(logits.shape, 9.0, dtype=probs_dtype, device="cuda")
    kda.kda_sample(logits.cuda(), u.cuda(), probs=out, **{k: v.cuda() for k, v in filters.items()})
    want = roll.sample(logits, u, **filters)[1]
    half = ref.HALF_STEP[torch.bfloat16] if probs_dtype == torch.bfloat16 else 0
    got = ref.np64(out)
    off = np.abs(got - want) - want * (half + 8 * 2.0 ** -24) - SMALLEST[probs_dtype]
    assert np.all(off <= 0), (float(off.max()), int(off.argmax()))
    return out


@pytest.mark.parametrize("probs_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("V", [37, 5000, 70001])
def test_masked_tokens_have_none(kda, V, dtype, probs_dtype):
    """Masked by the type's lowest value, by -1e9 or by -1e4: exactly zero, with temperature alone and with filters that keep everything."""
    gen = torch.Generator().manual_seed(V)
    logits, masked = torch.randn(3, V, generator=gen), torch.rand(3, V, generator=gen) < 0.6
    masked[:, V // 2] = False
    for n, value in enumerate((torch.finfo(dtype).min, -1e9, -1e4)):
        logits[n, masked[n]] = value
    logits, full = logits.to(dtype), lambda x: torch.full((3,), x)  # noqa: E731
    for filters in ({}, dict(temperature=full(0.7)), dict(temperature=full(3.0)), dict(min_p=full(1e-40)),
                    dict(top_k=torch.full((3,), V - 1, dtype=torch.int32)), dict(temperature=full(0.0))):
        out = _probs(kda, logits, probs_dtype, **filters)
        assert not bool(out.cpu()[masked].any())


@pytest.mark.parametrize("probs_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
@pytest.mark.parametrize("top", [0.0, 11.3, -300.0, 4096.0])
def test_unlikely_tokens_have_their_own(kda, top, dtype, probs_dtype):
    """Distances from the largest logit up to and beyond fp32's range, at several temperatures and places of the largest."""
    temperature = torch.tensor([1.0, 0.3, 2.5, 1.0, 40.0, 1e-3])
    steps = torch.linspace(0.0, 115.0, 3001)
    logits = top - temperature[:, None] * steps
    logits[3] = top - 2.0 ** torch.linspace(-20, 8, 3001)  # many close to it
    _probs(kda, logits.to(dtype), probs_dtype, temperature=temperature)
    # a first run of them, which top-k sorts
    _probs(kda, logits.to(dtype), probs_dtype, temperature=temperature, top_k=torch.full((6,), 1700, dtype=torch.int32))


def test_extreme_temperatures(kda):
    low = torch.finfo(torch.float32).min
    logits = torch.stack([torch.tensor([low, -low, 0.0, -1e38, 1e30]), torch.tensor([low, low, low, low, low]),
                          torch.tensor([3e38, -3e38, 2.9e38, 0.0, -float("inf")]), torch.tensor([1e-30, 0.0, -1e-30, 2e-30, -5e-29])])
    for t in (1e-29, 1e-6, 1.0, 1e30):
        _probs(kda, logits, torch.float32, temperature=torch.full((4,), t))


@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_temperatures_without_bound(kda, dtype):
    """Above 1e30 as at 1e30: ordinary logits are all alike, masked ones stay masked, whatever the row's largest is."""
    low, inf, V = torch.finfo(dtype).min, float("inf"), 3001
    gen = torch.Generator().manual_seed(3)
    logits = torch.randn(6, V, generator=gen)
    logits[1, 1::2] = low
    logits[2] = low                     # all of them masked alike
    logits[3] = low
    logits[3, ::3] = -inf
    logits[4] = -1e38
    logits[4, ::2] = -inf
    logits[5] *= 1e30
    logits, u = logits.to(dtype), torch.linspace(0.053, 0.951, 6)
    for t in (1e30, 3e36, 3e38, inf):
        temperature = torch.full((6,), t)
        for filters in ({}, dict(top_k=torch.full((6,), 500, dtype=torch.int32)), dict(top_p=torch.full((6,), 0.4)), dict(min_p=torch.full((6,), 0.5))):
            counts = dict(filters, temperature=temperature.clamp(max=1e30))
            want, p, margin = roll.sample(logits, u, **counts)
            kw = {k: v.cuda() for k, v in filters.items()}
            token, probs = kda.kda_sample(logits.cuda(), u.cuda(), temperature=temperature.cuda(), return_probs=True, **kw)
            assert np.array_equal(token.cpu().numpy(), want) and margin.min() > 1e-9
            assert np.all(np.abs(ref.np64(probs) - p) <= p * 8 * 2.0 ** -24 + 2.0 ** -149)
    _probs(kda, logits, torch.bfloat16, temperature=torch.full((6,), 1e30))


@pytest.mark.parametrize("V, depth", [((1 << 21) + 5, 25.0), ((1 << 21) + 5, 28.5), (1 << 19, 30.0), (1 << 24, 22.0)])
def test_long_tails(kda, V, depth):
    """One likely token and an equal tail far below it: a mass is good to 2e-10 of itself and half a unit, 2^-45 of the largest up to
    2^19 tokens and twice as much whenever there are twice as many, and so is what the draws go by."""
    half_unit = 2.0 ** -45 * 2.0 ** max(0, (V - 1).bit_length() - 19)
    logits = torch.full((1, V), -depth)
    logits[0, V // 3] = 0.0
    e = np.full(V, np.exp(-depth))
    e[V // 3] = 1.0
    upto = np.cumsum(e)
    slack = (2e-10 * upto[-1] + V * half_unit) * 2  # of the point and of the running mass
    dev = logits.cuda()
    for u in (1e-7, 3e-6, 0.5, 1 - 2.0 ** -16, 1 - 2.0 ** -20, 1 - 2.0 ** -24):
        token, probs = kda.kda_sample(dev, torch.tensor([u], device="cuda"), return_probs=True)
        i, point = int(token), float(np.float32(u)) * upto[-1]
        assert upto[i] > point - slack and (upto[i - 1] if i else 0.0) <= point + slack
    assert abs(float(probs.double().sum()) - 1) <= 8 * 2.0 ** -24 + slack
