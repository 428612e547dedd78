"""The speculative loop of the example: what it commits is what decoding the same tokens one by one commits."""
import os
import sys

import pytest
import torch

from tests._helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    ensure_built()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import spec_step
    return spec_step


def test_speculation_commits_what_decoding_commits(example):
    model, plain = example.HybridModel(seed=3), example.HybridModel(seed=3)
    one = torch.arange(model.N + 1, dtype=torch.int32, device="cuda")
    plain.root = model.root.clone()
    total = [0] * model.N
    streams = [[] for _ in total]
    for _ in range(6):
        counts = model.step()
        at = 0
        for n, c in enumerate(counts):
            streams[n] += model.last["tokens"][at:at + c].tolist()
            total[n] += c
            at += c
    assert model.ctx_len.tolist() == total and sum(total) > 6 * model.N and min(total) < 24  # some drafts accepted, some not
    # the same tokens, one per step and sequence, through the plain decode forms (sequences that have ended keep their state)
    import gated_linear_attention_chunk_gb300 as kda
    for t in range(max(total)):
        live = [n for n in range(model.N) if t < total[n]]
        tokens = torch.tensor([streams[n][t] if n in live else 0 for n in range(model.N)], dtype=torch.int32, device="cuda")
        _, (k, v, g, b), (ka, va) = plain.forward(tokens, one)
        keep = torch.tensor(live, device="cuda")
        cu = torch.tensor([sum(m < n for m in live) for n in range(model.N + 1)], dtype=torch.int32, device="cuda")
        kda.kda_replay_prep(plain.states, k[keep], v[keep], g[keep], b[keep], cu, plain.flags)
        plain.ctx_len = kda.kda_cache_append(ka, va, plain.k_pages, plain.v_pages, plain.table, plain.ctx_len, cu, rows=keep.int())
    assert plain.ctx_len.tolist() == total

    # matrix products of other shapes may round differently, by a few bf16 steps of the values they make
    def close(a, b):
        return float((a - b).norm() / b.norm()) < 0.02
    assert close(model.states, plain.states)
    for name in ("k_pages", "v_pages"):
        a, b = getattr(model, name).float(), getattr(plain, name).float()
        assert torch.equal(a == 0, b == 0) and close(a, b)  # the same rows written
