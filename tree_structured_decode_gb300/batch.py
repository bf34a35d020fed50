"""Python entry points of the operators whose lengths live on the GPU:
page tables and slot maps, the append by slot, attention behind a shared
prefix, and sampling.

Argument marshalling only: each function checks its tensors, makes the outputs
that were not given, and calls the C ABI (``include/tree_attn.h``).  The
functions take no host synchronisation and may be captured in a CUDA graph.
They run on the tensors' device: on ``stream`` if given, else on that device's
current stream.  What they allocate belongs to that stream; tensors made on
another one need the usual care (``wait_stream``, ``record_stream``).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

from ._abi import check, load_library

_NOTHING = contextlib.nullcontext()


@functools.lru_cache(maxsize=None)
def _codes():
    """tree_attn_dtype of torch's types."""
    import torch

    return {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _int32(name, x):
    """A number as the C ABI takes it: refused where ctypes would cut it to its low 32 bits."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def _index(name, t):
    """The CUDA device's index of a tensor."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _launch_on(index, stream):
    """(a context that makes the device and the stream current, the stream's handle)."""
    import torch

    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
        return (_NOTHING if index == torch._C._cuda_getDevice() else torch.cuda.device(index)), handle
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", index))
    if stream.device_index != index:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{index}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _vector(name, t, n, index, kind):
    """Address of a contiguous tensor of n elements."""
    if t.dtype is not kind or t.get_device() != index or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {kind} tensor of {n} on cuda:{index}, not {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _table(t, rows, index, kind):
    """Address, row stride and width of a block table."""
    if t.dtype is not kind or t.get_device() != index or t.dim() != 2:
        raise ValueError(f"block_table must be a 2-d {kind} tensor on cuda:{index}")
    n, width = t.shape
    _int32("block_table's width", width)
    stride = t.stride(0)
    if n != rows:
        raise ValueError(f"block_table has {n} rows for {rows} requests")
    if width > 1 and t.stride(1) != 1:
        raise ValueError("block_table must have contiguous rows")
    return t.data_ptr(), stride if rows > 1 and stride > width else width if rows <= 1 else stride, width


def _pools(k_pages, v_pages, index):
    """The pools' shape [pages, kv heads, 16, d], checked."""
    shape = k_pages.shape
    if _codes().get(k_pages.dtype, 2) > 1 or len(shape) != 4 or shape[2] != 16 or not k_pages.is_contiguous():
        raise ValueError("k_pages must be a contiguous bf16 or fp16 tensor [pages, kv heads, 16, d]")
    if (v_pages.dtype is not k_pages.dtype or v_pages.shape != shape or not v_pages.is_contiguous()
            or v_pages.get_device() != index or k_pages.get_device() != index):
        raise ValueError(f"v_pages must be as k_pages, {k_pages.dtype} {tuple(shape)}, both on cuda:{index}")
    return shape


def _rows(name, t, kind, d, index):
    """Shape and token stride of a [tokens, heads, d] tensor whose tokens are whole rows."""
    if t.dtype is not kind or t.get_device() != index or t.dim() != 3:
        raise ValueError(f"{name} must be a {kind} tensor [tokens, heads, {d}] on cuda:{index}")
    shape, (stride, head, one) = t.shape, t.stride()
    if shape[2] != d or one != 1 or (head != d and shape[1] > 1):
        raise ValueError(f"{name}: each token's [heads, {d}] must be contiguous")
    return shape, stride if shape[0] > 1 else shape[1] * d


def extend_tables(lens, n_new, block_table, free_pages, n_free, max_new, position_base=0, status=None, stream=None):
    """``tree_attn_extend_tables``: add ``n_new`` tokens to every request (negative: take back), in place.

    ``lens``, ``n_new`` int32 ``[requests]``; ``block_table`` int32 ``[requests, width]``; ``free_pages`` int32
    ``[capacity]`` with ``n_free`` int32 ``[1]`` (a stack); ``max_new`` the number of tokens that the outputs have room
    for.  Returns ``(slots, positions, cu_new)``, int32 ``[max_new]`` twice and ``[requests + 1]``.  All or nothing: see
    ``status`` (int32 ``[1]``, OR-ed) and ``include/tree_attn.h``."""
    import torch

    _int32("max_new", max_new), _int32("position_base", position_base)
    b, cap = _int32("lens' length", lens.numel()), _int32("free_pages' length", free_pages.numel())
    index, kind = _index("lens", lens), torch.int32
    table, stride, width = _table(block_table, b, index, kind)
    lens_at, new_at = _vector("lens", lens, b, index, kind), _vector("n_new", n_new, b, index, kind)
    free_at, n_free_at = _vector("free_pages", free_pages, cap, index, kind), _vector("n_free", n_free, 1, index, kind)
    status_at = None if status is None else _vector("status", status, 1, index, kind)
    if max_new < 0:
        raise ValueError("max_new is negative")
    context, handle = _launch_on(index, stream)
    with context:
        device = lens.device
        slots = torch.empty(max_new, dtype=kind, device=device)
        positions = torch.empty(max_new, dtype=kind, device=device)
        cu = torch.empty(b + 1, dtype=kind, device=device)
        check(load_library().tree_attn_extend_tables(
            lens_at, new_at, b, table, stride, width, free_at, cap, n_free_at, max_new, position_base, slots.data_ptr(),
            positions.data_ptr(), cu.data_ptr(), status_at, handle), "tree_attn_extend_tables")
    return slots, positions, cu


def append_slots(k_new, v_new, slots, k_pages, v_pages, status=None, stream=None):
    """``tree_attn_append_slots``: write ``k_new``, ``v_new`` (``[tokens, kv heads, d]``, each token's row contiguous) to
    ``slots`` (int32 ``[tokens]``, -1: none) of the page pools, in place."""
    import torch

    index, kind = _index("k_pages", k_pages), torch.int32
    pages, hkv, _, d = _pools(k_pages, v_pages, index)
    (t, h, _), ks = _rows("k_new", k_new, k_pages.dtype, d, index)
    shape, vs = _rows("v_new", v_new, k_pages.dtype, d, index)
    if h != hkv or shape[0] != t or shape[1] != hkv:
        raise ValueError(f"k_new {tuple(k_new.shape)} and v_new {tuple(v_new.shape)} must be [tokens, {hkv}, {d}]")
    slots_at = _vector("slots", slots, t, index, kind)
    status_at = None if status is None else _vector("status", status, 1, index, kind)
    context, handle = _launch_on(index, stream)
    with context:
        check(load_library().tree_attn_append_slots(
            k_new.data_ptr(), v_new.data_ptr(), ks, vs, slots_at, t, h, d, k_pages.data_ptr(), v_pages.data_ptr(),
            pages, status_at, handle), "tree_attn_append_slots")


@functools.lru_cache(maxsize=4096)
def _prefix_workspace(index, *sizes):
    """Bytes; by the sizes alone (on this device)."""
    need = ctypes.c_size_t(0)
    check(load_library().tree_attn_prefix_workspace(*sizes, ctypes.byref(need)), "tree_attn_prefix_workspace")
    return need.value


def prefix_attention(q, k_pages, v_pages, block_table, lens, cu_new=None, prefix_pages=None, prefix_len=0,
                     softmax_scale=0.0, out=None, lse=None, want_lse=True, status=None, stream=None):
    """``tree_attn_prefix_run``: every query attends to the shared prefix and to its own request's tokens.

    ``q`` ``[tokens, q heads, d]`` (each token's heads contiguous); ``block_table`` int32 ``[requests, width]`` and
    ``lens`` int32 ``[requests]`` as ``extend_tables`` keeps them; ``cu_new`` int32 ``[requests + 1]`` (None: one query a
    request); ``prefix_pages`` int32 with ``prefix_len`` tokens.  Returns ``(out, lse)``: ``out`` of q's type, ``lse``
    fp32 ``[tokens, q heads]`` (None without ``want_lse``)."""
    import torch

    _int32("prefix_len", prefix_len)
    index, kind, dtype = _index("q", q), torch.int32, q.dtype
    pages, hkv, _, d = _pools(k_pages, v_pages, index)
    if dtype is not k_pages.dtype:
        raise ValueError(f"q must be of the pools' type {k_pages.dtype}")
    (t, hq, _), q_stride = _rows("q", q, dtype, d, index)
    b = _int32("lens' length", lens.numel())
    table, stride, width = _table(block_table, b, index, kind)
    lens_at = _vector("lens", lens, b, index, kind)
    cu_at = None if cu_new is None else _vector("cu_new", cu_new, b + 1, index, kind)
    prefix_at = None
    if prefix_len > 0:
        if prefix_pages is None or prefix_pages.numel() * 16 < prefix_len:
            raise ValueError(f"prefix_pages holds fewer than prefix_len = {prefix_len} tokens")
        prefix_at = _vector("prefix_pages", prefix_pages, prefix_pages.numel(), index, kind)
    status_at = None if status is None else _vector("status", status, 1, index, kind)
    if out is not None:
        _vector("out", out, t * hq * d, index, dtype)
    if lse is not None:
        _vector("lse", lse, t * hq, index, torch.float32)
    context, handle = _launch_on(index, stream)
    with context:
        need = _prefix_workspace(index, b, t, prefix_len, hq, hkv, d)
        # from torch's allocator, call by call: runs on other streams or in other graphs have their own
        device = q.device
        work = torch.empty(need, dtype=torch.uint8, device=device)
        if out is None:
            out = torch.empty((t, hq, d), dtype=dtype, device=device)
        if lse is None and want_lse:
            lse = torch.empty((t, hq), dtype=torch.float32, device=device)
        check(load_library().tree_attn_prefix_run(
            q.data_ptr(), q_stride, k_pages.data_ptr(), v_pages.data_ptr(), pages, table, stride, width, lens_at, cu_at,
            b, t, prefix_at, prefix_len, hq, hkv, d, _codes()[dtype], softmax_scale, out.data_ptr(),
            None if lse is None else lse.data_ptr(), status_at, work.data_ptr(), need, handle), "tree_attn_prefix_run")
    return out, lse


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """``tree_attn_sample``: draw tokens from rows of logits with given random numbers.

    ``logits`` ``[rows, vocab]`` bf16, fp16 or fp32 (rows may lie apart); ``u`` fp32 in [0, 1), ``[rows]`` or ``[rows,
    draws]``: each number gives one token of its row.  ``temperature``, ``top_k``, ``top_p``, ``min_p``: one number for all
    rows, or a tensor ``[rows]`` (fp32; int32 for ``top_k``); None switches a filter off.  Returns ``(tokens, logprobs)``,
    int32 and fp32, shaped as ``u``; see ``include/tree_attn.h`` for the order of the filters and for rows that hold
    nothing to draw."""
    import torch

    if logits.numel() >= 2 ** 31 or u.numel() >= 2 ** 31:  # else no size of them is
        for n in (*logits.shape, *u.shape):
            _int32("a size of logits or u", n)
    index, real = _index("logits", logits), torch.float32
    code = _codes().get(logits.dtype)
    if code is None or logits.dim() != 2:
        raise ValueError("logits must be a bf16, fp16 or fp32 tensor [rows, vocab]")
    (rows, vocab), (stride, one) = logits.shape, logits.stride()
    if one != 1 and vocab > 1:
        raise ValueError("logits must have contiguous rows")
    shape = u.shape
    if len(shape) not in (1, 2) or shape[0] != rows:
        raise ValueError(f"u must be [{rows}] or [{rows}, draws], not {tuple(shape)}")
    u_at = _vector("u", u, u.numel(), index, real)
    draws = shape[1] if len(shape) == 2 else 1
    args = []
    for name, x, off, kind in (("temperature", temperature, 1.0, real), ("top_k", top_k, 0, torch.int32),
                               ("top_p", top_p, 1.0, real), ("min_p", min_p, 0.0, real)):
        if x is None:
            args += (None, off)
        elif isinstance(x, torch.Tensor):
            args += (_vector(name, x, rows, index, kind), off)
        else:
            x = type(off)(x)
            if kind is not real and not 0 <= x < vocab:
                x = 0  # such a top_k is off, and need not fit 32 bits
            args += (None, x)
    context, handle = _launch_on(index, stream)
    with context:
        device = logits.device
        tokens = torch.empty(shape, dtype=torch.int32, device=device)
        logprobs = torch.empty(shape, dtype=real, device=device)
        check(load_library().tree_attn_sample(
            logits.data_ptr(), stride if rows > 1 else vocab, code, rows, vocab, u_at, draws, *args, tokens.data_ptr(),
            logprobs.data_ptr(), handle), "tree_attn_sample")
    return tokens, logprobs
