"""Attention over a shared prefix: caches without pages or table columns, heads that fill more than a block, a capture as the first call."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import _rollout_reference as roll
from tests import _spec_reference as ref
from tests._helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


@pytest.mark.parametrize("pages, width", [(0, 0), (0, 3), (4, 0)])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_caches_without_pages_or_columns(kda, pages, width, dtype):
    """Empty prefixes leave the tail, or nothing; a row that no page holds is refused on the device."""
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, ot, lt = rand(5, 6, 64).to(dtype), rand(5, 6, 128).to(dtype), rand(5, 6)
    cu, none = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros(pages, 16, 2, d, device="cuda", dtype=dtype) for d in (64, 128))
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    o, lse = kda.kda_prefix_attn(q, kp, vp, table, none, cu)
    assert not o.any() and bool((lse == -float("inf")).all())
    o, lse = kda.kda_prefix_attn(q, kp, vp, table, none, cu, o_tail=ot, lse_tail=lt)
    assert torch.equal(o, ot) and torch.equal(lse, lt)
    ws = torch.full((kda.kda_prefix_attn_workspace_size(2, 5, 6, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    held = torch.full_like(ot, 3.0)
    kda.kda_prefix_attn(q, kp, vp, table, none + 1, cu, workspace=ws, o=held)
    assert kda.kda_device_status(ws) == kda.KDA_ERR_BAD_PAGE and bool((held == 3).all())


@pytest.mark.parametrize("G, Hkv, T, L", [(300, 1, 3, 200), (1000, 1, 1, 33), (257, 2, 2, 129), (4096, 1, 1, 20), (129, 1, 4, 300)])
@pytest.mark.parametrize("dtype", [ref.BF16, ref.F32])
def test_heads_of_one_token_beyond_a_block(kda, G, Hkv, T, L, dtype):
    kp, vp, table = ref.paged([L], 16, Hkv, 64, 64, dtype, 3)
    q = torch.randn(T, Hkv * G, 64, generator=torch.Generator().manual_seed(G)).to(dtype)
    cu, lens = torch.tensor([0, T], dtype=torch.int32), torch.tensor([L], dtype=torch.int32)
    o, lse = kda.kda_prefix_attn(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu.cuda())
    want = roll.prefix_attn(q, kp, vp, table, lens, cu, 64 ** -0.5)
    bo, bl = ref.attn_bounds(dtype, 64, L + 64, *want)
    assert np.all(np.abs(ref.np64(o) - want[0]) <= bo) and np.all(np.abs(ref.np64(lse) - want[1]) <= bl)


FIRST = """
import torch
import gated_linear_attention_chunk_gb300 as kda
dev, dt, n = "cuda", torch.{dtype}, {groups}
kp, vp = (torch.randn(8, 16, 2, 64, device=dev).to(dt) for _ in "kv")
table = torch.randint(0, 8, (n, 4), dtype=torch.int32, device=dev)
lens = torch.randint(0, 60, (n,), dtype=torch.int32, device=dev)
cu = torch.arange(n + 1, dtype=torch.int32, device=dev)
q = torch.randn(n, 4, 64, device=dev).to(dt)
freq, pos = torch.rand(32, dtype=torch.float64, device=dev), torch.arange(n, dtype=torch.int32, device=dev)
w, u = torch.ones(64, device=dev), torch.rand(n, device=dev)
def step():
    a, _ = kda.kda_norm_rope(q, None, pos, freq, w)
    o, lse = kda.kda_prefix_attn(a, kp, vp, table, lens, cu)
    g = kda.kda_norm_rope_bwd(q, None, o, None, pos, freq, w)
    return (o, lse, g[0], g[2], *kda.kda_sample(o.view(n, -1), u, return_probs=True))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
"""


@pytest.mark.parametrize("dtype, groups", [("bfloat16", 2), ("float32", 300)])
def test_the_first_call_of_a_process_is_captured(kda, dtype, groups):
    done = subprocess.run([sys.executable, "-c", FIRST.format(dtype=dtype, groups=groups)], capture_output=True, text=True, timeout=300,
                          cwd=__file__.rsplit("/tests/", 1)[0])
    assert done.returncode == 0, done.stderr[-2000:]
