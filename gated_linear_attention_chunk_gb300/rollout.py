"""A decoding step of branching rollouts (several samples of each prompt) in a hybrid model: binding of the calls.

    kda_norm_rope / kda_norm_rope_bwd   per-head norms of q and k with rotary positions, and the gradient
    kda_prefix_attn                     attention of a group of sequences over the prefix that they share
    kda_sample                          tokens (and distributions) from logits: temperature, top-k, top-p, min-p

They stand beside the speculative step (``spec.py``) and are bound in the same native module.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import kda as _kda
from .spec import _on, _spec


def kda_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                  mscale: float = 1.0, q_out=None, k_out=None,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """RMS norm of every head, times a weight, then rotary positions.  Returns ``(q_out, k_out)`` (k_out None for k None).

    q, k, positions, inv_freq, interleaved, mscale, q_out, k_out as for ``kda_rope``; q_weight, k_weight [d] (bf16 or fp32,
    both alike; None: ones).  ``kda_norm_rope(q, k, pos, w, wq, wk)`` is ``kda_rope`` of the normed heads, rounded once."""
    args = (q, k, None, None, positions, inv_freq, q_weight, k_weight, eps, interleaved, mscale, q_out, k_out, None, None, None)
    return _spec.norm_rope(*args) if stream is None else _on(stream, _spec.norm_rope, *args)


def kda_norm_rope_bwd_workspace_size(d: int) -> int:
    """Workspace of ``kda_norm_rope_bwd`` in bytes (0 for an invalid d)."""
    return int(_kda.load_library().kda_norm_rope_bwd_workspace_size(d))


def kda_norm_rope_bwd(q, k, d_q_out, d_k_out, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                      interleaved: bool = False, mscale: float = 1.0, d_q=None, d_k=None, d_q_weight=None, d_k_weight=None,
                      workspace=None, stream=None):
    """Gradient of ``kda_norm_rope``.  Returns ``(d_q, d_k, d_q_weight, d_k_weight)``.

    q, k are the forward's inputs, d_q_out, d_k_out the gradients of its outputs (tokens may be strided).  The weights'
    gradients are fp32 [d], None where no weight (and no output for it) is given."""
    if d_q_out is None:
        raise TypeError("d_q_out must be a torch.Tensor")
    args = (q, k, d_q_out, d_k_out, positions, inv_freq, q_weight, k_weight, eps, interleaved, mscale, d_q, d_k, d_q_weight,
            d_k_weight, workspace)
    return _spec.norm_rope(*args) if stream is None else _on(stream, _spec.norm_rope, *args)


def kda_prefix_attn_workspace_size(N: int, T: int, Hq: int, Hkv: int, dv: int) -> int:
    """Workspace of ``kda_prefix_attn`` in bytes (0 for invalid arguments)."""
    return int(_kda.load_library().kda_prefix_attn_workspace_size(N, T, Hq, Hkv, dv))


def kda_prefix_attn(q, k_pages, v_pages, block_table, prefix_len, cu_tokens, scale: Optional[float] = None, o_tail=None, lse_tail=None,
                    o=None, lse=None, return_lse: bool = True, workspace=None,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of N groups of sequences over each group's shared prefix.  Returns ``(o [T, Hq, dv], lse [T, Hq] fp32 or None)``.

    q [T, Hq, dk] (tokens may be strided), packed group by group: group g has the tokens cu_tokens[g] : cu_tokens[g + 1] of its
    sequences; k_pages, v_pages as for ``kda_tree_attn``, block_table [N, max_pages] and prefix_len [N] int32: the groups'
    prefixes.  Every token attends to all of its group's prefix, which is read once for all of them.  With ``o_tail`` [T, Hq, dv]
    and ``lse_tail`` [T, Hq], the result of ``kda_tree_attn`` over each sequence's own keys, ``(o, lse)`` are the attention
    over both.  ``o`` and ``lse`` may be the tail's tensors.  ``scale`` defaults to dk ** -0.5."""
    args = (q, k_pages, v_pages, block_table, prefix_len, cu_tokens, scale, o_tail, lse_tail, o, lse, return_lse, workspace)
    return _spec.prefix_attn(*args) if stream is None else _on(stream, _spec.prefix_attn, *args)


def kda_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, return_probs: bool = False, token=None, probs=None,
               stream=None):
    """Tokens drawn from logits [N, V] (bf16 or fp32; rows may be strided) by given uniforms u [N] fp32.

    Per row, each [N] or None: ``temperature`` fp32 (0: the largest logit; at most 1e30), ``top_k`` int32 (0: off), ``top_p`` fp32 (1: off),
    ``min_p`` fp32 (0: off), applied in this order; ties go to the lower index, and the token is the lowest kept index whose
    running mass exceeds u of the whole.  Returns token [N] int32 (-1 for a row without a finite logit), or ``(token, probs)``
    with ``return_probs`` or an output ``probs`` [N, V] (fp32, or the given tensor's bf16): the distribution that the token was
    drawn from, as ``kda_draft_verify`` takes it."""
    args = (logits, u, temperature, top_k, top_p, min_p, return_probs, token, probs)
    return _spec.sample(*args) if stream is None else _on(stream, _spec.sample, *args)
