"""Python entry points of the operators whose lengths live on the GPU:
page tables and slot maps, the append by slot, attention behind a shared
prefix, and sampling.

Argument marshalling only: each function checks its tensors, makes the outputs
that were not given, and calls the C ABI (``include/tree_attn.h``).  The
functions take no host synchronisation and may be captured in a CUDA graph.
They run on the tensors' device: on ``stream`` if given, else on that device's
current stream.
"""
from __future__ import annotations

import contextlib
import ctypes

from ._abi import check, load_library

_DTYPE = None


def _dtype(t):
    global _DTYPE
    if _DTYPE is None:
        import torch

        _DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    return _DTYPE.get(t.dtype, -1)


def _launch_on(device, stream):
    """(a context that makes `device` and `stream` current, the stream's handle)."""
    import torch

    index = device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
        if index == torch.cuda.current_device():
            return contextlib.nullcontext(), handle
        return torch.cuda.device(index), handle
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _ints(name, t, shape, device):
    import torch

    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {shape}")
    return t.data_ptr()


def _status(t, device):
    return None if t is None else _ints("status", t, (1,), device)


def _table(t, rows, device):
    import torch

    if t.dtype != torch.int32 or t.device != device or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"block_table must be a 2-d int32 tensor on {device} with contiguous rows")
    if t.shape[0] != rows:
        raise ValueError(f"block_table has {t.shape[0]} rows for {rows} requests")
    stride = t.stride(0) if rows > 1 else t.shape[1]
    return t.data_ptr(), max(stride, t.shape[1]) if rows <= 1 else stride, t.shape[1]


def _cuda(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _pools(k_pages, v_pages, device):
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if _dtype(t) not in (0, 1) or t.device != device or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous bf16 or fp16 tensor [pages, kv heads, 16, d] on {device}")
    if k_pages.dtype != v_pages.dtype or k_pages.shape != v_pages.shape or k_pages.shape[2] != 16:
        raise ValueError("k_pages and v_pages must have one type and one shape [pages, kv heads, 16, d]")


def _rows(name, t, pools):
    """Token stride of a [tokens, heads, d] tensor whose tokens are whole rows."""
    if t.dtype != pools.dtype or t.device != pools.device or t.dim() != 3:
        raise ValueError(f"{name} must be a [tokens, heads, d] tensor of the pools' type and device")
    n, h, d = t.shape
    if d != pools.shape[3] or t.stride(2) != 1 or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: each token's [heads, d={pools.shape[3]}] must be contiguous")
    return t.stride(0) if n > 1 else h * d


def extend_tables(lens, n_new, block_table, free_pages, n_free, max_new, position_base=0, status=None, stream=None):
    """``tree_attn_extend_tables``: add ``n_new`` tokens to every request (negative: take back), in place.

    ``lens``, ``n_new`` int32 ``[requests]``; ``block_table`` int32 ``[requests, width]``; ``free_pages`` int32
    ``[capacity]`` with ``n_free`` int32 ``[1]`` (a stack); ``max_new`` the number of tokens that the outputs have room
    for.  Returns ``(slots, positions, cu_new)``, int32 ``[max_new]`` twice and ``[requests + 1]``.  All or nothing: see
    ``status`` (int32 ``[1]``, OR-ed) and ``include/tree_attn.h``."""
    import torch

    device = _cuda("lens", lens)
    b = lens.shape[0]
    table, stride, width = _table(block_table, b, device)
    args = (_ints("lens", lens, (b,), device), _ints("n_new", n_new, (b,), device), b, table, stride, width,
            _ints("free_pages", free_pages, (free_pages.numel(),), device), free_pages.numel(),
            _ints("n_free", n_free, (1,), device))
    max_new = int(max_new)
    if max_new < 0:
        raise ValueError("max_new is negative")
    context, handle = _launch_on(device, stream)
    with context:
        # one allocation: slots, positions, cu_new
        out = torch.empty(2 * max_new + b + 1, dtype=torch.int32, device=device)
        slots, positions, cu = out.split_with_sizes((max_new, max_new, b + 1))
        at = out.data_ptr()
        check(load_library().tree_attn_extend_tables(*args, max_new, int(position_base), at, at + 4 * max_new,
                                                     at + 8 * max_new, _status(status, device), handle),
              "tree_attn_extend_tables")
    return slots, positions, cu


def append_slots(k_new, v_new, slots, k_pages, v_pages, status=None, stream=None):
    """``tree_attn_append_slots``: write ``k_new``, ``v_new`` (``[tokens, kv heads, d]``, each token's row contiguous) to
    ``slots`` (int32 ``[tokens]``, -1: none) of the page pools, in place."""
    device = _cuda("k_pages", k_pages)
    _pools(k_pages, v_pages, device)
    ks, vs = _rows("k_new", k_new, k_pages), _rows("v_new", v_new, k_pages)
    t, h, d = k_new.shape
    if k_new.shape != v_new.shape or h != k_pages.shape[1]:
        raise ValueError(f"k_new {tuple(k_new.shape)} and v_new {tuple(v_new.shape)} must be "
                         f"[tokens, {k_pages.shape[1]}, {d}]")
    slots_at = _ints("slots", slots, (t,), device)
    context, handle = _launch_on(device, stream)
    with context:
        check(load_library().tree_attn_append_slots(k_new.data_ptr(), v_new.data_ptr(), ks, vs, slots_at, t, h, d,
                                                    k_pages.data_ptr(), v_pages.data_ptr(), k_pages.shape[0],
                                                    _status(status, device), handle), "tree_attn_append_slots")


def prefix_attention(q, k_pages, v_pages, block_table, lens, cu_new=None, prefix_pages=None, prefix_len=0,
                     softmax_scale=0.0, out=None, lse=None, want_lse=True, status=None, stream=None):
    """``tree_attn_prefix_run``: every query attends to the shared prefix and to its own request's tokens.

    ``q`` ``[tokens, q heads, d]`` (each token's heads contiguous); ``block_table`` int32 ``[requests, width]`` and
    ``lens`` int32 ``[requests]`` as ``extend_tables`` keeps them; ``cu_new`` int32 ``[requests + 1]`` (None: one query a
    request); ``prefix_pages`` int32 with ``prefix_len`` tokens.  Returns ``(out, lse)``: ``out`` of q's type, ``lse``
    fp32 ``[tokens, q heads]`` (None without ``want_lse``)."""
    import torch

    device = _cuda("q", q)
    _pools(k_pages, v_pages, device)
    q_stride = _rows("q", q, k_pages)
    t, hq, d = q.shape
    b = lens.shape[0]
    table, stride, width = _table(block_table, b, device)
    lens_at = _ints("lens", lens, (b,), device)
    cu_at = None if cu_new is None else _ints("cu_new", cu_new, (b + 1,), device)
    prefix_len, prefix_at = int(prefix_len), None
    if prefix_pages is not None:
        prefix_at = _ints("prefix_pages", prefix_pages, (prefix_pages.numel(),), device)
    if prefix_len > 0 and (prefix_pages is None or prefix_pages.numel() * 16 < prefix_len):
        raise ValueError(f"prefix_pages holds fewer than prefix_len = {prefix_len} tokens")
    for name, x, shape, dtype in (("out", out, (t, hq, d), q.dtype), ("lse", lse, (t, hq), torch.float32)):
        if x is not None and (x.dtype != dtype or x.device != device or not x.is_contiguous() or tuple(x.shape) != shape):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {device}")
    lib = load_library()
    context, handle = _launch_on(device, stream)
    with context:
        need = ctypes.c_size_t(0)
        check(lib.tree_attn_prefix_workspace(b, t, prefix_len, hq, k_pages.shape[1], d, ctypes.byref(need)),
              "tree_attn_prefix_workspace")
        # from torch's allocator, call by call: runs on other streams or in other graphs have their own
        work = torch.empty(need.value, dtype=torch.uint8, device=device)
        if out is None:
            out = torch.empty((t, hq, d), dtype=q.dtype, device=device)
        if lse is None and want_lse:
            lse = torch.empty((t, hq), dtype=torch.float32, device=device)
        check(lib.tree_attn_prefix_run(q.data_ptr(), q_stride, k_pages.data_ptr(), v_pages.data_ptr(), k_pages.shape[0],
                                       table, stride, width, lens_at, cu_at, b, t, prefix_at, prefix_len, hq,
                                       k_pages.shape[1], d, _dtype(q), float(softmax_scale), out.data_ptr(),
                                       None if lse is None else lse.data_ptr(), _status(status, device), work.data_ptr(),
                                       need.value, handle), "tree_attn_prefix_run")
    return out, lse


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """``tree_attn_sample``: draw tokens from rows of logits with given random numbers.

    ``logits`` ``[rows, vocab]`` bf16, fp16 or fp32 (rows may lie apart); ``u`` fp32 in [0, 1), ``[rows]`` or ``[rows,
    draws]``: each number gives one token of its row.  ``temperature``, ``top_k``, ``top_p``, ``min_p``: one number for all
    rows, or a tensor ``[rows]`` (fp32; int32 for ``top_k``); None switches a filter off.  Returns ``(tokens, logprobs)``,
    int32 and fp32, shaped as ``u``; see ``include/tree_attn.h`` for the order of the filters and for rows that hold
    nothing to draw."""
    import torch

    device = _cuda("logits", logits)
    code = _dtype(logits)
    if code < 0 or logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a bf16, fp16 or fp32 tensor [rows, vocab] with contiguous rows")
    rows, vocab = logits.shape
    if u.dtype != torch.float32 or u.device != device or not u.is_contiguous() or u.dim() not in (1, 2) or u.shape[0] != rows:
        raise ValueError(f"u must be a contiguous fp32 tensor [{rows}] or [{rows}, draws] on {device}")
    draws = u.shape[1] if u.dim() == 2 else 1
    args = []
    for name, x, off, kind in (("temperature", temperature, 1.0, torch.float32), ("top_k", top_k, 0, torch.int32),
                               ("top_p", top_p, 1.0, torch.float32), ("min_p", min_p, 0.0, torch.float32)):
        if isinstance(x, torch.Tensor):
            if x.dtype != kind or x.device != device or not x.is_contiguous() or x.dim() != 1 or x.shape[0] != rows:
                raise ValueError(f"{name} must be a number or a contiguous {kind} tensor [{rows}] on {device}")
            args += [x.data_ptr(), off]
        else:
            args += [None, off if x is None else type(off)(x)]
    context, handle = _launch_on(device, stream)
    with context:
        tokens = torch.empty(u.shape, dtype=torch.int32, device=device)
        logprobs = torch.empty(u.shape, dtype=torch.float32, device=device)
        check(load_library().tree_attn_sample(logits.data_ptr(), logits.stride(0) if rows > 1 else vocab, code, rows, vocab,
                                              u.data_ptr(), draws, *args, tokens.data_ptr(), logprobs.data_ptr(), handle),
              "tree_attn_sample")
    return tokens, logprobs
