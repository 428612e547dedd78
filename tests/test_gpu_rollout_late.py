"""Late inputs (test_gpu_rollout_order.py) for the calls' other ways: top-k, greedy and min-p rows, and more groups than the attention's kernels
plan themselves."""
import pytest
import torch

from tests._helpers import ensure_built

pytestmark = pytest.mark.gpu

LATE = 2_000_000  # clocks: about a millisecond


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as g
    return g


def _operators(kda, dtype):
    g = torch.Generator("cuda").manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    N, Hq, Hkv, d, page = 300, 4, 2, 64, 16
    table = torch.randperm(2 * N, generator=g, device="cuda").to(torch.int32).view(N, 2)
    lens = torch.randint(0, 33, (N,), generator=g, device="cuda", dtype=torch.int32)
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    pool, rows = (2 * N, page, Hkv, d), torch.rand(5, generator=g, device="cuda")
    zeros = torch.zeros(5, device="cuda")
    return [
        ([rand(N, Hq, d), rand(*pool), rand(*pool), table, lens, cu, rand(N, Hq, d), rand(N, Hq).float()],
         lambda q, k, v, t, n, c, o, m: kda.kda_prefix_attn(q, k, v, t, n, c, o_tail=o, lse_tail=m)),
        ([rand(5, 9001), rows, ints(1, 7, 500, 3000, 20)], lambda x, u, k: kda.kda_sample(x, u, top_k=k, return_probs=True)),
        ([rand(5, 9001), rows, zeros], lambda x, u, t: kda.kda_sample(x, u, temperature=t, return_probs=True)),
        ([rand(5, 9001), rows, rows / 8], lambda x, u, m: kda.kda_sample(x, u, min_p=m, return_probs=True)),
    ]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("captured", [False, True])
def test_late_inputs(kda, dtype, captured):
    stream = torch.cuda.Stream()
    for good, call in _operators(kda, dtype):
        want = [x.clone() for x in call(*good)]
        late, out = [x.clone() for x in good], []

        def run():
            torch.cuda._sleep(LATE)
            for x, y in zip(late, good):
                torch.add(y, 0, out=x)
            out[:] = call(*late)

        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            if captured:
                call(*good)  # (allocations and the first launch)
                stream.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    run()
            for x in late:
                x.zero_()
            graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [16, 17, 256, 257, 600])
def test_plans_of_any_size_follow_one_another(kda, N, dtype):
    """Calls of different batches through one workspace, back to back, against each with a workspace of its own: the plan that lies there is
    written by every CTA, or by a launch ahead of them."""
    g = torch.Generator("cuda").manual_seed(N)
    Hq, Hkv, d, page = 4, 2, 64, 16
    kp, vp = (torch.randn(64, page, Hkv, d, generator=g, device="cuda").to(dtype) for _ in "kv")
    cases = []
    for n in (N, 3, N - 1, 1):
        table = torch.randint(0, 64, (n, 8), generator=g, device="cuda", dtype=torch.int32)
        lens = torch.randint(0, 8 * page + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        tokens = torch.randint(0, 4, (n,), generator=g, device="cuda")
        tokens[0] += 1
        cu = torch.cat([tokens.new_zeros(1), tokens.cumsum(0)]).int()
        cases.append((torch.randn(int(cu[-1]), Hq, d, generator=g, device="cuda").to(dtype), kp, vp, table, lens, cu))
    need = max(kda.kda_prefix_attn_workspace_size(len(c[4]), len(c[0]), Hq, Hkv, d) for c in cases)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    want = [kda.kda_prefix_attn(*c) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [kda.kda_prefix_attn(*c, workspace=ws) for c in cases]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
