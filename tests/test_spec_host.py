"""The speculative-step calls without a GPU: refusals on the host, workspace sizes, the frequency table."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests._helpers import ensure_built

FAKE = 0x10000  # a 16-byte aligned non-null value; never dereferenced (the checks fail first)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    import gated_linear_attention_chunk_gb300 as m
    return m


class _PagedKV(ctypes.Structure):
    _fields_ = [(x, ctypes.c_void_p) for x in ("k", "v")] + [(x, ctypes.c_int64) for x in (
        "k_page_stride", "k_row_stride", "k_head_stride", "v_page_stride", "v_row_stride", "v_head_stride", "num_pages",
        "table_stride")] + [(x, ctypes.c_void_p) for x in ("block_table", "ctx_len")] + [
        (x, ctypes.c_int) for x in ("page_size", "max_pages")]


def _cache(kda, **kw):
    f = dict(k=FAKE, v=FAKE, k_page_stride=16 * 1024, k_row_stride=1024, k_head_stride=128, v_page_stride=16 * 1024,
             v_row_stride=1024, v_head_stride=128, num_pages=8, table_stride=4, block_table=FAKE, ctx_len=FAKE, page_size=16,
             max_pages=4)
    f.update(kw)
    return ctypes.byref(_PagedKV(**f))


def test_codes_and_names(kda):
    assert kda.kda_status_string(kda.KDA_ERR_BAD_PAGE) == "KDA_ERR_BAD_PAGE"
    assert kda.kda_status_string(kda.KDA_ERR_BAD_TREE) == "KDA_ERR_BAD_TREE"


@pytest.mark.parametrize("name", ["kda_rope", "kda_rope_bwd"])
def test_rope_refusals(kda, name):
    f = getattr(kda.load_library(), name)
    base = dict(q=FAKE, k=FAKE, dtype=0, pos=FAKE, w=FAKE, T=4, Hq=8, Hk=2, d=128, rot=128, qs=0, ks=0, inter=0, m=1.0,
                qo=FAKE, ko=FAKE, qos=0, kos=0, stream=None)
    call = lambda **kw: f(*({**base, **kw}).values())  # noqa: E731
    assert call(dtype=3) == UNSUPPORTED
    assert call(d=100) == UNSUPPORTED and call(d=2048) == UNSUPPORTED
    for bad in (dict(rot=130), dict(rot=63), dict(rot=-2), dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(q=None), dict(qo=None),
                dict(pos=None), dict(w=None), dict(ko=None), dict(q=FAKE + 1), dict(pos=FAKE + 2), dict(w=FAKE + 4),
                dict(qs=1023), dict(kos=255)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, q=None, qo=None) == OK  # nothing to do: nothing is launched


def test_tree_attn_refusals(kda):
    lib = kda.load_library()
    big = 1 << 40
    base = dict(q=FAKE, k=FAKE, v=FAKE, dtype=0, cache=_cache(kda), cu=FAKE, parent=None, N=2, T=8, Hq=8, Hkv=2, dk=128, dv=128,
                qs=0, ks=0, vs=0, nodes=4, scale=1.0, o=FAKE, lse=None, ws=FAKE, wsb=big, stream=None)
    call = lambda **kw: lib.kda_tree_attn(*({**base, **kw}).values())  # noqa: E731
    assert call(dtype=2) == UNSUPPORTED and call(dk=96) == UNSUPPORTED and call(dv=256) == UNSUPPORTED
    for bad in (dict(Hq=9), dict(Hkv=0), dict(N=-1), dict(T=-1), dict(nodes=0), dict(nodes=65), dict(T=9), dict(q=None),
                dict(v=None), dict(o=None), dict(cu=None), dict(cu=FAKE + 2), dict(q=FAKE + 8), dict(qs=1020), dict(ks=248),
                dict(cache=None), dict(cache=_cache(kda, page_size=0)), dict(cache=_cache(kda, k_row_stride=1025)),
                dict(cache=_cache(kda, k=None)), dict(cache=_cache(kda, v=FAKE + 2)), dict(cache=_cache(kda, ctx_len=None)),
                dict(cache=_cache(kda, block_table=None)), dict(cache=_cache(kda, table_stride=3)),
                dict(cache=_cache(kda, page_size=1 << 20, max_pages=1 << 12, table_stride=1 << 12))):
        assert call(**bad) == INVALID, bad
    need = kda.kda_tree_attn_workspace_size(2, 8, 8, 2, 128, 4, 64)
    assert need > 256
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE
    assert kda.kda_tree_attn_workspace_size(2, 8, 9, 2, 128, 4, 64) == 0
    assert kda.kda_tree_attn_workspace_size(2, 8, 8, 2, 96, 4, 64) == 0
    # a longer context has more parts, up to the number that fills the GPU
    sizes = [kda.kda_tree_attn_workspace_size(2, 8, 8, 2, 128, 4, c) for c in (64, 4096, 1 << 20, 1 << 24)]
    assert sizes[0] < sizes[1] < sizes[2] == sizes[3]


def test_append_refusals(kda):
    lib = kda.load_library()
    base = dict(k=FAKE, v=FAKE, dtype=0, cache=_cache(kda), cu=FAKE, rows=None, N=2, A=8, T=8, Hkv=8, dk=128, dv=128, ks=0, vs=0,
                new=FAKE + 64, ws=FAKE, wsb=256, stream=None)
    call = lambda **kw: lib.kda_cache_append(*({**base, **kw}).values())  # noqa: E731
    assert call(dk=32) == UNSUPPORTED and call(dtype=-1) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(wsb=255) == WORKSPACE
    for bad in (dict(A=9), dict(A=-1), dict(T=-1), dict(Hkv=0), dict(k=None), dict(v=FAKE + 4), dict(cu=None), dict(ks=1023),
                dict(new=FAKE), dict(new=FAKE + 1), dict(rows=FAKE + 1), dict(cache=_cache(kda, v_head_stride=4))):
        assert call(**bad) == INVALID, bad


def test_verify_refusals(kda):
    lib = kda.load_library()
    need = kda.kda_draft_verify_workspace_size(2)
    assert need == 256 + 16
    base = dict(tokens=FAKE, cu=FAKE, parent=None, p=FAKE, q=FAKE, dtype=1, ua=FAKE, us=FAKE, N=2, T=8, V=100, ts=0, ds=0,
                cua=FAKE, rows=FAKE, nxt=FAKE, ws=FAKE, wsb=need, stream=None)
    call = lambda **kw: lib.kda_draft_verify(*({**base, **kw}).values())  # noqa: E731
    assert call(dtype=9) == UNSUPPORTED and call(V=(1 << 24) + 1) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE
    for bad in (dict(V=0), dict(N=-1), dict(T=-1), dict(ts=99), dict(ds=99), dict(tokens=None), dict(cu=None), dict(p=None),
                dict(ua=None), dict(us=None), dict(cua=None), dict(rows=None), dict(nxt=None), dict(p=FAKE + 2),
                dict(tokens=FAKE + 1)):
        assert call(**bad) == INVALID, bad


def test_python_checks(kda):
    """The binding refuses tensors that are not on the GPU before any call."""
    x, pos, w = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        kda.kda_rope(x, None, pos, w)
    with pytest.raises(TypeError):
        kda.kda_rope([1.0], None, pos, w)
    with pytest.raises(ValueError):
        kda.kda_draft_verify(pos, pos, torch.zeros(2, 5), torch.zeros(2), torch.zeros(1))


def test_rope_frequencies(kda):
    f = lambda *a, **k: kda.rope_frequencies(*a, device="cpu", **k)  # noqa: E731
    w, m = f(64)
    assert m == 1.0 and w.dtype == torch.float64
    np.testing.assert_allclose(w.numpy(), [10000.0 ** (-2 * j / 64) for j in range(32)], rtol=1e-15)
    lin, _ = f(64, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin.numpy(), w.numpy() / 4, rtol=1e-15)
    ntk, _ = f(64, scaling="ntk", factor=4.0)  # the fastest pair stays, the slowest is divided by the factor
    assert ntk[0] == 1.0 and math.isclose(float(ntk[-1]), float(w[-1]) / 4, rel_tol=1e-12)
    yarn, m = f(64, scaling="yarn", factor=4.0, original_len=4096)
    assert m == pytest.approx(0.1 * math.log(4.0) + 1)
    turns = 4096 * w / (2 * math.pi)
    assert torch.equal(yarn[turns > 64], w[turns > 64])       # well above beta_fast turns: kept
    np.testing.assert_allclose(yarn[turns < 0.5].numpy(), w[turns < 0.5].numpy() / 4, rtol=1e-15)
    assert bool((yarn[1:] < yarn[:-1]).all())
    assert f(0)[0].numel() == 0
    for bad in (dict(rot=63), dict(rot=64, scaling="other"), dict(rot=64, factor=0.0)):
        with pytest.raises(ValueError):
            f(**bad)


def test_reference_verification_keeps_the_target_distribution():
    """The walk's definition itself: over many uniforms, the first token after the root follows the target's row, whatever
    the draft's (repeated rejection sampling; two children drawn from the draft, in exact expectation over a grid)."""
    from tests import _spec_reference as ref
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    got = np.zeros(3)
    grid = (np.arange(24) + 0.5) / 24
    for x1 in range(3):
        for x2 in range(3):
            for u1 in grid:
                for u2 in grid:
                    probs = torch.tensor(np.stack([p, p, p]))
                    draft = torch.tensor(np.stack([q, q, q]))
                    args = (torch.tensor([0, x1, x2]), [0, 3], torch.tensor([-1, 0, 0]), probs, draft, torch.tensor([0, u1, u2]))
                    weight = q[x1] * q[x2] / len(grid) ** 2
                    cu, rows, nxt = ref.verify(*args, torch.tensor([0.5]))
                    if cu[1] == 2:  # a child stands: it is the first token
                        got[[x1, x2][rows[1] - 1]] += weight
                    else:           # otherwise the draw, integrated over its own number
                        for us in grid:
                            got[ref.verify(*args, torch.tensor([us]))[2][0]] += weight / len(grid)
    np.testing.assert_allclose(got, p, atol=3 / len(grid))


def test_reference_ancestors():
    from tests import _spec_reference as ref
    sees = ref.ancestors([-1, 0, 0, 1, 3, 2])
    assert [list(np.flatnonzero(r)) for r in sees] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [0, 2, 5]]
