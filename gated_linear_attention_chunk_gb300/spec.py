"""One speculative step of the softmax-attention layers beside KDA layers: binding of the calls.

    kda_rope / kda_rope_bwd   rotary positions of q and k, and the gradient
    kda_tree_attn             drafted trees attend to a paged cache and to their own ancestors
    kda_draft_verify          which drafted tokens stand, and the next token
    kda_cache_append          rows (a prompt's, or the accepted nodes') into the paged cache

``rope_frequencies`` makes the frequency table of ``kda_rope`` (plain, or scaled for long contexts).
The accepted nodes go on to ``kda_replay`` for the recurrent states: ``cu_accept`` is its argument, and
``rows`` picks the tokens' k, v, g and beta.  Like the rest of the package the functions check their
tensors, allocate what was not passed and call the C entry point of the same name on a stream.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import Optional, Tuple

import torch

from . import kda as _kda
from .kda import KDA_BF16, KDA_F32, KDA_WS_HEADER_BYTES, KdaError

KDA_MAX_TREE_NODES = 64

_CODES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}


class _PagedKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_page_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_page_stride", ctypes.c_int64), ("v_row_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p),
                ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int)]


_raw_stream = torch._C._cuda_getCurrentRawStream  # (torch.cuda.current_stream builds an object around it)
_capturing = torch.cuda.is_current_stream_capturing


def _code(t: torch.Tensor, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has unsupported dtype {t.dtype} (bf16 or fp32)")
    return code


def _token_stride(t, name: str, dtype, H: int, d: int, T: Optional[int] = None) -> int:
    """Checks a [T, H, d] tensor whose tokens may be strided (a slice of a fused projection); its token stride."""
    try:
        n, h, e = t.shape
        if t.dtype is dtype and t.is_cuda and h == H and e == d and (T is None or n == T):
            s0, s1, s2 = t.stride()
            if s2 == 1 and (s1 == d or H == 1):
                if n <= 1:
                    return 0
                if s0 >= H * d:
                    return s0
                raise ValueError(f"{name} must not have overlapping tokens (stride {s0} < {H * d})")
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    except ValueError as e:
        if str(e).startswith(name):
            raise
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 3 or t.shape[1:] != (H, d) or (T is not None and t.shape[0] != T):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({'T' if T is None else T}, {H}, {d})")
    raise ValueError(f"{name} must have contiguous tokens (only its first dimension may be strided)")


def _ints(t, name: str, n: Optional[int] = None):
    """Checks a contiguous int32 CUDA vector and returns its address (None for None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != 1 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA vector")
    if n is not None and shape[0] != n:
        raise ValueError(f"{name} has {shape[0]} entries, expected {n}")
    return t.data_ptr()


def _on(device, stream, call):
    """``call(handle)`` with the tensors' device current, on the given stream or the current one; what it allocates
    belongs to that stream."""
    index = device.index
    if stream is None:
        if index == torch.cuda.current_device():
            return call(_raw_stream(index))
        with torch.cuda.device(device):
            return call(_raw_stream(index))
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _check(rc: int, where: str):
    if rc:
        raise KdaError(rc, where)


_KEEP_BYTES = 64 << 20  # scratch up to this size is kept for the next call
_scratch = threading.local()


def _workspace(workspace, nbytes: int, device, handle):
    """The caller's workspace, or scratch: ``(address, bytes, owner)``.

    Scratch is one buffer per thread, device and stream, since the calls on a stream run one after the other; it grows, and holds
    nothing from call to call.  Calls that a graph records, and large ones, get a buffer of their own."""
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if nbytes <= _KEEP_BYTES and not _capturing():
        kept = _scratch.__dict__
        key = (device.index, handle)
        entry = kept.get(key)
        if entry is None or entry[1] < nbytes:
            size = max(nbytes, 1 << 16)
            buf = torch.empty((size,), dtype=torch.uint8, device=device)
            entry = kept[key] = (buf.data_ptr(), size, buf)
        return entry
    buf = torch.empty((nbytes,), dtype=torch.uint8, device=device)
    return buf.data_ptr(), nbytes, buf


def _cache(k_pages, v_pages, block_table, ctx_len, dtype, Hkv: int, dk: int, dv: int) -> Tuple[_PagedKV, int, int]:
    """The checked cache as its C struct; the number of sequences, and the rows that a block table can name."""
    for name, t, d in (("k_pages", k_pages, dk), ("v_pages", v_pages, dv)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        shape = t.shape
        if not t.is_cuda or t.dtype is not dtype or len(shape) != 4 or t.stride(3) != 1:
            raise ValueError(f"{name} must be a CUDA tensor [pages, page_size, Hkv, d] of {dtype} with contiguous channels")
        if shape[2] != Hkv or shape[3] != d:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected [pages, page_size, {Hkv}, {d}]")
    pages, page, _, _ = k_pages.shape
    if v_pages.shape[0] != pages or v_pages.shape[1] != page:
        raise ValueError("k_pages and v_pages must have the same pages and page size")
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda or block_table.dtype is not torch.int32 \
            or block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be an int32 CUDA matrix [N, max_pages] with contiguous rows")
    N, max_pages = block_table.shape
    k0, k1, k2, _ = k_pages.stride()
    v0, v1, v2, _ = v_pages.stride()
    return _PagedKV(k_pages.data_ptr(), v_pages.data_ptr(), k0, k1, k2, v0, v1, v2, pages,
                    block_table.stride(0) if N > 1 else max_pages, block_table.data_ptr(), _ints(ctx_len, "ctx_len", N), page,
                    max_pages), N, page * max_pages


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
    return _rope("kda_rope", q, k, positions, inv_freq, interleaved, mscale, q_out, k_out, stream)


def kda_rope_bwd(d_q_out, d_k_out, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, d_q=None,
                 d_k=None, stream=None):
    """Gradient of ``kda_rope``: from the gradients of its outputs to those of q and k.  Returns ``(d_q, d_k)``."""
    return _rope("kda_rope_bwd", d_q_out, d_k_out, positions, inv_freq, interleaved, mscale, d_q, d_k, stream)


def _rope(name, q, k, positions, inv_freq, interleaved, mscale, q_out, k_out, stream):
    lib = _kda.load_library()
    T, Hq, d = q.shape
    dt, code = q.dtype, _code(q, "q")
    qs = _token_stride(q, "q", dt, Hq, d)
    Hk, ks = 0, 0
    if k is not None:
        Hk = k.shape[1]
        ks = _token_stride(k, "k", dt, Hk, d, T)
    pos = _ints(positions, "positions", T)
    if inv_freq.dtype is not torch.float64 or not inv_freq.is_cuda or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous fp64 CUDA vector")

    def call(handle):
        qo = torch.empty((T, Hq, d), dtype=dt, device=q.device) if q_out is None else q_out
        qos = 0 if q_out is None else _token_stride(q_out, "q_out", dt, Hq, d, T)
        if k is None:
            ko, kos, kp, kop = None, 0, None, None
        else:
            ko = torch.empty((T, Hk, d), dtype=dt, device=q.device) if k_out is None else k_out
            kos = 0 if k_out is None else _token_stride(k_out, "k_out", dt, Hk, d, T)
            kp, kop = k.data_ptr(), ko.data_ptr()
        _check(getattr(lib, name)(q.data_ptr(), kp, code, pos, inv_freq.data_ptr(), T, Hq, Hk, d, 2 * inv_freq.shape[0], qs, ks,
                                  bool(interleaved), mscale, qo.data_ptr(), kop, qos, kos, handle), name)
        return qo, ko

    return _on(q.device, stream, call)


def kda_tree_attn_workspace_size(N: int, T: int, Hq: int, Hkv: int, dv: int, max_nodes: int, max_ctx: int) -> int:
    """Workspace of ``kda_tree_attn`` in bytes (0 for invalid arguments); max_ctx = block-table columns x page size."""
    return int(_kda.load_library().kda_tree_attn_workspace_size(N, T, Hq, Hkv, dv, max_nodes, max_ctx))


def kda_tree_attn(q, k, v, k_pages, v_pages, block_table, ctx_len, cu_nodes, parent=None, scale: Optional[float] = None,
                  max_nodes: int = KDA_MAX_TREE_NODES, o=None, lse=None, return_lse: bool = True, workspace=None,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of drafted trees over a paged cache.  Returns ``(o [T, Hq, dv], lse [T, Hq] fp32 or None)``.

    q [T, Hq, dk]; k [T, Hkv, dk], v [T, Hkv, dv]: the nodes' own keys and values (tokens may be strided); k_pages
    [pages, page_size, Hkv, dk], v_pages [.., dv] (any axis order with contiguous channels); block_table [N, max_pages],
    ctx_len [N], cu_nodes [N+1], parent [T] int32 (None: chains).  A node attends to its sequence's first ctx_len cache
    rows, its ancestors and itself; one-node trees are the plain decode step.  ``scale`` defaults to dk ** -0.5;
    ``max_nodes`` bounds the trees of the batch."""
    lib = _kda.load_library()
    T, Hq, dk = q.shape
    Hkv, dv = v.shape[1], v.shape[2]
    dt, code = q.dtype, _code(q, "q")
    qs = _token_stride(q, "q", dt, Hq, dk)
    ks, vs = _token_stride(k, "k", dt, Hkv, dk, T), _token_stride(v, "v", dt, Hkv, dv, T)
    cache, N, max_ctx = _cache(k_pages, v_pages, block_table, ctx_len, dt, Hkv, dk, dv)
    cu, par = _ints(cu_nodes, "cu_nodes", N + 1), _ints(parent, "parent", T)
    if o is not None:
        _kda._need(o, "o", dt, (T, Hq, dv))
    if lse is not None:
        _kda._need(lse, "lse", torch.float32, (T, Hq))

    def call(handle):
        dev = q.device
        out = torch.empty((T, Hq, dv), dtype=dt, device=dev) if o is None else o
        sums = torch.empty((T, Hq), dtype=torch.float32, device=dev) if lse is None and return_lse else lse
        need = 0  # (0 for sizes that the call itself refuses)
        if workspace is None:
            need = lib.kda_tree_attn_workspace_size(N, T, Hq, Hkv, dv, max_nodes, max_ctx) or KDA_WS_HEADER_BYTES
        ws, size, _ = _workspace(workspace, need, dev, handle)
        _check(lib.kda_tree_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), code, ctypes.byref(cache), cu, par, N, T, Hq, Hkv, dk,
                                 dv, qs, ks, vs, max_nodes, dk ** -0.5 if scale is None else scale, out.data_ptr(),
                                 None if sums is None else sums.data_ptr(), ws, size, handle), "kda_tree_attn")
        return out, sums

    return _on(q.device, stream, call)


def kda_cache_append(k, v, k_pages, v_pages, block_table, ctx_len, cu, rows=None, new_len=None, workspace=None,
                     stream=None) -> torch.Tensor:
    """Rows j in [cu[n], cu[n+1]) go to the positions after ctx_len[n] of sequence n.  Returns the new lengths [N].

    Row j is row ``rows[j]`` of k [T, Hkv, dk] and v [T, Hkv, dv], or row j itself; ``kda_draft_verify``'s cu_accept and
    rows append the accepted nodes.  Rows from cu[N] on are not read.  The pools are written in place."""
    lib = _kda.load_library()
    T, Hkv, dk = k.shape
    dv = v.shape[2]
    dt, code = k.dtype, _code(k, "k")
    ks, vs = _token_stride(k, "k", dt, Hkv, dk), _token_stride(v, "v", dt, Hkv, dv, T)
    cache, N, _ = _cache(k_pages, v_pages, block_table, ctx_len, dt, Hkv, dk, dv)
    c, r = _ints(cu, "cu", N + 1), _ints(rows, "rows")

    def call(handle):
        new = torch.empty((N,), dtype=torch.int32, device=k.device) if new_len is None else new_len
        ws, size, _ = _workspace(workspace, KDA_WS_HEADER_BYTES, k.device, handle)
        _check(lib.kda_cache_append(k.data_ptr(), v.data_ptr(), code, ctypes.byref(cache), c, r, N,
                                    T if rows is None else rows.shape[0], T, Hkv, dk, dv, ks, vs,
                                    _ints(new, "new_len", N), ws, size, handle),
               "kda_cache_append")
        return new

    return _on(k.device, stream, call)


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
    lib = _kda.load_library()
    T, V = target_probs.shape
    N = cu_nodes.shape[0] - 1
    code = _code(target_probs, "target_probs")
    for name, t in (("target_probs", target_probs), ("draft_probs", draft_probs)):
        if t is not None and (not t.is_cuda or t.dtype is not target_probs.dtype or t.shape != (T, V)
                              or (V > 1 and t.stride(1) != 1)):
            raise ValueError(f"{name} must be a CUDA matrix [{T}, {V}] of {target_probs.dtype} with contiguous rows")
    for name, t, n in (("u_accept", u_accept, T), ("u_sample", u_sample, N)):
        if not t.is_cuda or t.dtype is not torch.float32 or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA vector of {n}")
    tok, cu, par = _ints(tokens, "tokens", T), _ints(cu_nodes, "cu_nodes"), _ints(parent, "parent", T)
    dev = target_probs.device

    def call(handle):
        if cu_accept is None and rows is None and next_token is None:  # one allocation for the three
            counts, packed, nxt = torch.empty((2 * N + 1 + T,), dtype=torch.int32, device=dev).split((N + 1, T, N))
        else:
            counts = torch.empty((N + 1,), dtype=torch.int32, device=dev) if cu_accept is None else cu_accept
            packed = torch.empty((T,), dtype=torch.int32, device=dev) if rows is None else rows
            nxt = torch.empty((N,), dtype=torch.int32, device=dev) if next_token is None else next_token
        ws, size, _ = _workspace(workspace, KDA_WS_HEADER_BYTES + 8 * N, dev, handle)
        q, qs = (None, 0) if draft_probs is None else (draft_probs.data_ptr(), draft_probs.stride(0) if T > 1 else 0)
        _check(lib.kda_draft_verify(tok, cu, par, target_probs.data_ptr(), q, code, u_accept.data_ptr(), u_sample.data_ptr(), N, T,
                                    V, target_probs.stride(0) if T > 1 else 0, qs, _ints(counts, "cu_accept", N + 1),
                                    _ints(packed, "rows", T), _ints(nxt, "next_token", N), ws, size, handle),
               "kda_draft_verify")
        return counts, packed, nxt

    return _on(dev, stream, call)
