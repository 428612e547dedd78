"""One speculative step of the softmax-attention layers beside KDA layers: binding of the calls.

    kda_rope / kda_rope_bwd   rotary positions of q and k, and the gradient
    kda_tree_attn             drafted trees attend to a paged cache and to their own ancestors
    kda_draft_verify          which drafted tokens stand, and the next token
    kda_cache_append          rows (a prompt's, or the accepted nodes') into the paged cache

``rope_frequencies`` makes the frequency table of ``kda_rope`` (plain, or scaled for long contexts).
The accepted nodes go on to ``kda_replay`` for the recurrent states: ``cu_accept`` is its argument, and
``rows`` picks the tokens' k, v, g and beta (their number, ``cu_accept[-1]``, has to be read on the host for that).  Like the rest of the package the functions check their
tensors, allocate what was not passed and call the C entry point of the same name on a stream; the checks and the
call are in ``_lib/_spec.so`` (``csrc/spec_binding.cpp``), since on small inputs they would take longer than the kernels.
"""
from __future__ import annotations

import importlib.util
import math
import os
from typing import Optional, Tuple

import torch

from . import kda as _kda

KDA_MAX_TREE_NODES = 64

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "_spec.so")


def _load_binding():
    if not os.path.exists(BINDING_PATH):
        raise ImportError(f"_spec.so is not built ({BINDING_PATH}); run __graft_entry__.build()")
    _kda.load_library()
    spec = importlib.util.spec_from_file_location("gated_linear_attention_chunk_gb300._lib._spec", BINDING_PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


_spec = _load_binding()


def _on(stream, call, *args):
    """``call(*args)`` on a stream: what it allocates belongs to that stream."""
    with torch.cuda.stream(stream):
        return call(*args)


def rope_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device="cuda") -> Tuple[torch.Tensor, float]:
    """The table of ``kda_rope``: ``(inv_freq [rot/2] fp64, mscale)``.

    ``scaling`` extends the context by ``factor``: "linear" divides every frequency, "ntk" enlarges the base so that
    the slowest pair is divided by ``factor`` and the fastest stays, "yarn" keeps the pairs that turn more than
    ``beta_fast`` times over ``original_len`` positions, divides those that turn less than ``beta_slow`` times, ramps
    between, and returns mscale = 0.1 ln(factor) + 1."""
    if rot < 0 or rot % 2:
        raise ValueError(f"rot must be even and not negative, got {rot}")
    if base <= 0 or factor <= 0:
        raise ValueError("base and factor must be positive")
    j = torch.arange(0, rot, 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    w = base ** (-j / rot) if rot else j
    if scaling == "linear":
        w = w / factor
    elif scaling == "yarn" and rot:
        def pair(turns):  # the pair that turns that often over the original length
            return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
        ramp = ((j / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        w = w / factor * ramp + w * (1 - ramp)
        mscale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "none", "ntk", "linear", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return w.to(device), mscale


def kda_rope(q, k, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, q_out=None, k_out=None,
             stream=None):
    """Rotary positions.  Returns ``(q_out, k_out)`` (k_out None for k None).

    q [T, Hq, d], k [T, Hk, d] (bf16 or fp32; tokens may be strided); positions [T] int32; inv_freq [rot/2] fp64,
    rot <= d (the other channels are copied).  Pairs are (j, j + rot/2), or (2j, 2j+1) with ``interleaved``; rotated values
    are multiplied by ``mscale``.  ``q_out`` / ``k_out`` may be q / k themselves."""
    args = (False, q, k, positions, inv_freq, interleaved, mscale, q_out, k_out)
    return _spec.rope(*args) if stream is None else _on(stream, _spec.rope, *args)


def kda_rope_bwd(d_q_out, d_k_out, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, d_q=None,
                 d_k=None, stream=None):
    """Gradient of ``kda_rope``: from the gradients of its outputs to those of q and k.  Returns ``(d_q, d_k)``."""
    args = (True, d_q_out, d_k_out, positions, inv_freq, interleaved, mscale, d_q, d_k)
    return _spec.rope(*args) if stream is None else _on(stream, _spec.rope, *args)


def kda_tree_attn_workspace_size(N: int, T: int, Hq: int, Hkv: int, dv: int, max_nodes: int, max_ctx: int,
                                 dtype: Optional[torch.dtype] = None) -> int:
    """Workspace of ``kda_tree_attn`` in bytes (0 for invalid arguments); max_ctx = block-table columns x page size.
    ``dtype`` bf16 or fp32: what that type needs; None: enough for either."""
    lib = _kda.load_library()
    if dtype is None:
        return int(lib.kda_tree_attn_workspace_size(N, T, Hq, Hkv, dv, max_nodes, max_ctx))
    code = {torch.bfloat16: _kda.KDA_BF16, torch.float32: _kda.KDA_F32}.get(dtype, -1)
    return int(lib.kda_tree_attn_workspace_size_for(code, N, T, Hq, Hkv, dv, max_nodes, max_ctx))


def kda_tree_attn(q, k, v, k_pages, v_pages, block_table, ctx_len, cu_nodes, parent=None, scale: Optional[float] = None,
                  max_nodes: int = KDA_MAX_TREE_NODES, o=None, lse=None, return_lse: bool = True, workspace=None,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of drafted trees over a paged cache.  Returns ``(o [T, Hq, dv], lse [T, Hq] fp32 or None)``.

    q [T, Hq, dk]; k [T, Hkv, dk], v [T, Hkv, dv]: the nodes' own keys and values (tokens may be strided); k_pages
    [pages, page_size, Hkv, dk], v_pages [.., dv] (any axis order with contiguous channels); block_table [N, max_pages],
    ctx_len [N], cu_nodes [N+1], parent [T] int32 (None: chains).  A node attends to its sequence's first ctx_len cache
    rows, its ancestors and itself; one-node trees are the plain decode step.  ``scale`` defaults to dk ** -0.5;
    ``max_nodes`` bounds the trees of the batch; pass the real bound where it is known (it sizes the workspace, and above
    32 rows per KV head adds two launches)."""
    args = (q, k, v, k_pages, v_pages, block_table, ctx_len, cu_nodes, parent, scale, max_nodes, o, lse, return_lse, workspace)
    return _spec.tree_attn(*args) if stream is None else _on(stream, _spec.tree_attn, *args)


def kda_cache_append(k, v, k_pages, v_pages, block_table, ctx_len, cu, rows=None, new_len=None, workspace=None,
                     stream=None) -> torch.Tensor:
    """Rows j in [cu[n], cu[n+1]) go to the positions after ctx_len[n] of sequence n.  Returns the new lengths [N].

    Row j is row ``rows[j]`` of k [T, Hkv, dk] and v [T, Hkv, dv], or row j itself; ``kda_draft_verify``'s cu_accept and
    rows append the accepted nodes.  Rows from cu[N] on are not read.  The pools are written in place.  After BAD_SLOT, or
    BAD_PAGE of a row, a new length covers a row that was not written."""
    args = (k, v, k_pages, v_pages, block_table, ctx_len, cu, rows, new_len, workspace)
    return _spec.cache_append(*args) if stream is None else _on(stream, _spec.cache_append, *args)


def kda_draft_verify_workspace_size(N: int) -> int:
    """Workspace of ``kda_draft_verify`` in bytes."""
    return int(_kda.load_library().kda_draft_verify_workspace_size(N))


def kda_draft_verify(tokens, cu_nodes, target_probs, u_accept, u_sample, parent=None, draft_probs=None, cu_accept=None,
                     rows=None, next_token=None, workspace=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Verification of drafted trees.  Returns ``(cu_accept [N+1], rows [T], next_token [N])``, int32.

    tokens [T], cu_nodes [N+1], parent [T] int32 (None: chains); target_probs [T, V] (bf16 or fp32; rows may be
    strided): the target's distribution after each node; draft_probs [T, V]: the distribution each node's children were
    drawn from (None: drafts taken as certain); u_accept [T], u_sample [N] fp32 uniforms in [0, 1).  Sequence n accepts
    the packed nodes rows[cu_accept[n] : cu_accept[n+1]], the root first; next_token[n] follows them."""
    args = (tokens, cu_nodes, target_probs, u_accept, u_sample, parent, draft_probs, cu_accept, rows, next_token, workspace)
    return _spec.draft_verify(*args) if stream is None else _on(stream, _spec.draft_verify, *args)
