"""Python entry points of the operators that take prompts in and verify trees of
drafted tokens: attention of several new tokens a request, the drafts that
stand, their keys and values moved together, and scores of tokens.

Argument marshalling only, as in ``batch.py``: each function checks its tensors,
makes the outputs, and calls the C ABI (``include/tree_attn.h``).  The functions
take no host synchronisation and may be captured in a CUDA graph; they run on the
tensors' device, on ``stream`` if given, else on that device's current stream.
"""
from __future__ import annotations

import ctypes
import functools

from ._abi import check, load_library
from .batch import _codes, _index, _int32, _launch_on, _pools, _rows, _table, _vector


@functools.lru_cache(maxsize=4096)
def _chunk_workspace(index, *sizes):
    """Bytes; by the sizes alone (on this device)."""
    need = ctypes.c_size_t(0)
    check(load_library().tree_attn_chunk_workspace(*sizes, ctypes.byref(need)), "tree_attn_chunk_workspace")
    return need.value


def _chunk(q, k_pages, v_pages, block_table, lens, parents, cu_new, softmax_scale, out, lse, want_lse, status, stream):
    import torch

    index, kind, dtype = _index("q", q), torch.int32, q.dtype
    pages, hkv, _, d = _pools(k_pages, v_pages, index)
    if dtype is not k_pages.dtype:
        raise ValueError(f"q must be of the pools' type {k_pages.dtype}")
    (t, hq, _), q_stride = _rows("q", q, dtype, d, index)
    _int32("q's tokens", t)
    b = _int32("lens' length", lens.numel())
    table, stride, width = _table(block_table, b, index, kind)
    lens_at = _vector("lens", lens, b, index, kind)
    cu_at = None if cu_new is None else _vector("cu_new", cu_new, b + 1, index, kind)
    parents_at = None if parents is None else _vector("parents", parents, t, index, kind)
    status_at = None if status is None else _vector("status", status, 1, index, kind)
    if out is not None:
        _vector("out", out, t * hq * d, index, dtype)
    if lse is not None:
        _vector("lse", lse, t * hq, index, torch.float32)
    context, handle = _launch_on(index, stream)
    with context:
        need = _chunk_workspace(index, b, t, hq, hkv, d)
        # from torch's allocator, call by call: runs on other streams or in other graphs have their own
        device = q.device
        work = torch.empty(need, dtype=torch.uint8, device=device)
        if out is None:
            out = torch.empty((t, hq, d), dtype=dtype, device=device)
        if lse is None and want_lse:
            lse = torch.empty((t, hq), dtype=torch.float32, device=device)
        check(load_library().tree_attn_chunk_run(
            q.data_ptr(), q_stride, k_pages.data_ptr(), v_pages.data_ptr(), pages, table, stride, width, lens_at, cu_at,
            parents_at, b, t, hq, hkv, d, _codes()[dtype], softmax_scale, out.data_ptr(),
            None if lse is None else lse.data_ptr(), status_at, work.data_ptr(), need, handle), "tree_attn_chunk_run")
    return out, lse


def prompt_attention(q, k_pages, v_pages, block_table, lens, cu_new=None, softmax_scale=0.0, out=None, lse=None,
                     want_lse=True, status=None, stream=None):
    """``tree_attn_chunk_run`` without parents: causal attention of prompts, or chunks of them, of different lengths.

    ``q`` ``[tokens, q heads, d]`` (each token's heads contiguous), packed: request b's new tokens are ``cu_new[b]`` to
    ``cu_new[b + 1]`` (int32 ``[requests + 1]``; None: one each).  Their keys and values are in the pools already:
    ``block_table`` and ``lens`` as ``extend_tables`` keeps them, this step's tokens counted.  New token i of n sees its
    request's first ``lens[b] - n + i + 1`` tokens.  Returns ``(out, lse)``: ``out`` of q's type, ``lse`` fp32 ``[tokens, q
    heads]`` (None without ``want_lse``)."""
    return _chunk(q, k_pages, v_pages, block_table, lens, None, cu_new, softmax_scale, out, lse, want_lse, status, stream)


def draft_attention(q, k_pages, v_pages, block_table, lens, parents, cu_new=None, softmax_scale=0.0, out=None, lse=None,
                    want_lse=True, status=None, stream=None):
    """``tree_attn_chunk_run`` with parents: attention of a tree of drafted tokens of each request over its cache.

    As ``prompt_attention``, but new token i of n sees the first ``lens[b] - n`` tokens of its request, itself, and the new
    tokens above it: ``parents`` int32 ``[tokens]`` has the one right above, counted within the request and below i, or -1.
    At most 128 new tokens a request."""
    if parents is None:
        raise ValueError("parents must be an int32 tensor [tokens]")
    return _chunk(q, k_pages, v_pages, block_table, lens, parents, cu_new, softmax_scale, out, lse, want_lse, status, stream)


def accept_drafts(drafted, parents, cu_new, sampled, status=None, stream=None):
    """``tree_attn_accept_drafts``: which drafts agree with the tokens that the model drew at the nodes.

    ``drafted``, ``parents``, ``sampled`` int32 ``[tokens]``; ``cu_new`` int32 ``[requests + 1]``.  Node 0 of a request is
    kept, and of a kept node's children the first whose drafted token was drawn there.  Returns ``(path, n_kept,
    next_tokens, n_back)``: ``path`` int32 ``[tokens]``, the kept nodes of request b from ``cu_new[b]`` on and -1 behind
    them; the others int32 ``[requests]``; ``n_back`` (kept - nodes) is for ``extend_tables``."""
    import torch

    index, kind = _index("drafted", drafted), torch.int32
    t = _int32("drafted's length", drafted.numel())
    if cu_new.numel() < 1:
        raise ValueError("cu_new must be [requests + 1]")
    b = _int32("cu_new's length", cu_new.numel()) - 1
    at = [_vector(name, x, t, index, kind) for name, x in (("drafted", drafted), ("parents", parents), ("sampled", sampled))]
    cu_at = _vector("cu_new", cu_new, b + 1, index, kind)
    status_at = None if status is None else _vector("status", status, 1, index, kind)
    context, handle = _launch_on(index, stream)
    with context:
        device = drafted.device
        path = torch.empty(t, dtype=kind, device=device)
        kept = torch.empty(b, dtype=kind, device=device)
        following = torch.empty(b, dtype=kind, device=device)
        back = torch.empty(b, dtype=kind, device=device)
        check(load_library().tree_attn_accept_drafts(
            at[0], at[1], cu_at, at[2], b, t, path.data_ptr(), kept.data_ptr(), following.data_ptr(), back.data_ptr(),
            status_at, handle), "tree_attn_accept_drafts")
    return path, kept, following, back


def _layers(k_pages, v_pages, index):
    """(layers, pages, kv heads, d, elements from one layer's pool to the next) of a pool or of all layers' pools, checked."""
    if k_pages.dim() != 5:
        pages, hkv, _, d = _pools(k_pages, v_pages, index)
        return 1, pages, hkv, d, 0
    shape = k_pages.shape
    if v_pages.shape != shape or v_pages.stride() != k_pages.stride():
        raise ValueError(f"v_pages must be as k_pages, {tuple(shape)}")
    layers = _int32("the number of layers", shape[0])
    if layers == 0:
        return 0, 0, 0, 0, 0
    pages, hkv, _, d = _pools(k_pages[0], v_pages[0], index)
    between = k_pages.stride(0)
    if layers > 1 and between < pages * hkv * 16 * d:
        raise ValueError("the layers' pools must lie one behind another")
    return layers, pages, hkv, d, between if layers > 1 else 0


def keep_drafts(path, cu_new, block_table, lens, k_pages, v_pages, status=None, stream=None):
    """``tree_attn_keep_drafts``: move the kept nodes' keys and values together, in place.

    ``path``, ``cu_new`` as of ``accept_drafts``; ``lens`` still counts all nodes.  ``k_pages``, ``v_pages``: a pool ``[pages,
    kv heads, 16, d]``, or the pools of all layers ``[layers, pages, kv heads, 16, d]``, moved in one launch."""
    import torch

    index, kind = _index("k_pages", k_pages), torch.int32
    layers, pages, hkv, d, between = _layers(k_pages, v_pages, index)
    if layers == 0:
        return
    b = _int32("lens' length", lens.numel())
    t = _int32("path's length", path.numel())
    table, stride, width = _table(block_table, b, index, kind)
    path_at, lens_at = _vector("path", path, t, index, kind), _vector("lens", lens, b, index, kind)
    cu_at = _vector("cu_new", cu_new, b + 1, index, kind)
    status_at = None if status is None else _vector("status", status, 1, index, kind)
    context, handle = _launch_on(index, stream)
    with context:
        check(load_library().tree_attn_keep_drafts(
            path_at, cu_at, lens_at, table, stride, width, b, t, k_pages.data_ptr(), v_pages.data_ptr(), between, layers, pages, hkv,
            d, status_at, handle), "tree_attn_keep_drafts")


def token_logprobs(logits, tokens=None, temperature=1.0, top=0, stream=None):
    """``tree_attn_token_logprobs``: log probabilities of given tokens, entropy, and the likeliest tokens.

    ``logits`` ``[rows, vocab]`` bf16, fp16 or fp32 (rows may lie apart); ``tokens`` int32 ``[rows]`` or ``[rows, n]``, or
    None; ``temperature`` one number for all rows, or fp32 ``[rows]``.  Returns ``(logprobs, entropy, top_tokens,
    top_logprobs)``: fp32 shaped as ``tokens`` (None without), fp32 ``[rows]``, and int32 and fp32 ``[rows, top]``; see
    ``include/tree_attn.h`` for masked and broken rows."""
    import torch

    if logits.numel() >= 2 ** 31:  # else no size of it is
        for n in logits.shape:
            _int32("a size of logits", n)
    _int32("top", top)
    if top < 0:
        raise ValueError("top is negative")
    index, kind, real = _index("logits", logits), torch.int32, torch.float32
    code = _codes().get(logits.dtype)
    if code is None or logits.dim() != 2:
        raise ValueError("logits must be a bf16, fp16 or fp32 tensor [rows, vocab]")
    (rows, vocab), (stride, one) = logits.shape, logits.stride()
    if one != 1 and vocab > 1:
        raise ValueError("logits must have contiguous rows")
    n_given, given_at = 0, None
    if tokens is not None:
        shape = tokens.shape
        if len(shape) not in (1, 2) or shape[0] != rows:
            raise ValueError(f"tokens must be [{rows}] or [{rows}, n], not {tuple(shape)}")
        n_given = _int32("tokens a row", shape[1]) if len(shape) == 2 else 1
        given_at = _vector("tokens", tokens, rows * n_given, index, kind)
    if isinstance(temperature, torch.Tensor):
        heat, heat_all = _vector("temperature", temperature, rows, index, real), 1.0
    else:
        heat, heat_all = None, 1.0 if temperature is None else float(temperature)
    context, handle = _launch_on(index, stream)
    with context:
        device = logits.device
        given = None if tokens is None else torch.empty(shape, dtype=real, device=device)
        entropy = torch.empty(rows, dtype=real, device=device)
        best = torch.empty((rows, top), dtype=kind, device=device)
        best_logprobs = torch.empty((rows, top), dtype=real, device=device)
        check(load_library().tree_attn_token_logprobs(
            logits.data_ptr(), stride if rows > 1 else vocab, code, rows, vocab, given_at, n_given, heat, heat_all, top,
            None if given is None else given.data_ptr(), entropy.data_ptr(), best.data_ptr(), best_logprobs.data_ptr(),
            handle), "tree_attn_token_logprobs")
    return given, entropy, best, best_logprobs
