"""The operators between the projection's rows and the cache: norm of queries and keys with
their rotation by position, attention of whole prompts, and a paged cache in 4 bits with its
append, its reading and the attention of drafted trees over it.

Marshalling only, as in _ops: every argument is checked here, outputs and the workspace come
from torch's allocator on the current stream, and the library's kernels do the rest on that
stream. The formulas, and what happens to out-of-range values on the device, stand in
include/tf_exl3.h. None of these calls has a gradient: where autograd follows an input, the
results are part of its graph, and a backward pass that reaches them raises; with out=, a call is
refused where autograd follows an input or the buffer. The cache takes values: to autograd its
rows are constants.
"""

from __future__ import annotations

import struct

from . import _lib
from ._lib import _dt_code, _run, _torch, load
from ._ops import (
    _ATTENTION,
    _changed,
    _floats,
    _followed,
    _halves,
    _need,
    _nodes,
    _one_gpu,
    _pack,
    _ptr,
    _refuse_followed,
    _whole,
    _workspace,
)

_ROTATE = struct.Struct("@10if8P13q")
_PROMPT = struct.Struct("@6if5P8q")
_APPEND = struct.Struct("@8i8P13q")
_READ = struct.Struct("@8i7P13q")


def q4_row_bytes(dim: int) -> int:
    """Bytes of a row of dim numbers in 4 bits, 5 * dim / 8 (tf_exl3_q4_row_bytes); dim a multiple of 32."""
    if dim < 32 or dim % 32 or dim > 1 << 24:
        raise ValueError(f"rows in 4 bits have a multiple of 32 numbers, not {dim}")
    return dim // 8 * 5


def _without_gradient(name, result, *inputs):
    return _nodes()[0].apply(name, result, *inputs)


# ---------------------------------------------------------------- norm and rotation


def _check_norm_rotate(q, k, positions, frequencies, q_weight, k_weight, outs):
    torch = _torch()
    _need("q", q, q.dim() if q is not None and q.dim() in (3, 4) else 4, _floats())
    *tokens, heads, dim = q.shape
    same = (q.dtype,)
    _need("k", k, len(tokens) + 2, same, (*tokens, None, dim))
    if frequencies is not None:
        _need("frequencies", frequencies, 1, (torch.float32,))
        _need("positions", positions, len(tokens), (torch.int32,), tuple(tokens))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _need(name, w, 1, _floats(), (dim,))
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError(f"q_weight and k_weight must have one element type, not {q_weight.dtype} and {k_weight.dtype}")
    for name, o, x in zip(("q_out", "k_out"), outs, (q, k)):
        if o is not None:
            _need(name, o, x.dim(), same, tuple(x.shape))
    _one_gpu(q, k, positions if frequencies is not None else None, frequencies, q_weight, k_weight, *outs)


def _is_weight(torch, w, dtype, dim, device):
    return (
        (dtype is torch.bfloat16 or dtype is torch.float16 or dtype is torch.float32) and w.dtype is dtype
        and w.shape == (dim,) and w.is_contiguous() and w.get_device() == device
    )


def _pair(out):
    if len(out) != 2:
        raise ValueError("out must be a pair of tensors")
    return out


def norm_rotate(q, k, positions, frequencies, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, out=None):
    """(q', k'): each head's row divided by its root mean square, times the weight, and turned by
    its token's position (tf_exl3_norm_rotate).

    q [batch][tokens][q_heads][dim] and k [batch][tokens][kv_heads][dim] of fp32, fp16 or bf16 with
    positions int32 [batch][tokens], or all three without the batch: packed tokens. Views of a
    fused projection's rows will do. frequencies fp32 [rotary_dim / 2], radians a position
    (rotary_dim a multiple of 8 from 16 up to dim); the pairs are (f, f + rotary_dim / 2), or (2f, 2f + 1)
    where interleaved; None turns nothing (positions are not looked at). q_weight, k_weight [dim], None for ones. eps None: no norm,
    and no weights. out: the pair of results, which may be (q, k) themselves; refused where autograd
    follows any of the tensors."""
    torch = _torch()
    q_out, k_out = (None, None) if out is None else _pair(out)
    if eps is None and not (q_weight is None and k_weight is None):
        raise ValueError("weights belong to the norm: eps is None")
    dev = -1
    try:
        shape, rows, t, d = q.shape, k.shape, q.dtype, q.get_device()
        dim, tokens = shape[-1], shape[:-2]
        w = k_weight if q_weight is None else q_weight
        if (
            (t is torch.bfloat16 or t is torch.float16 or t is torch.float32) and k.dtype is t
            and (len(shape) == 4 or len(shape) == 3) and rows[:-2] == tokens and rows[-1] == dim
            and q.stride(-1) == k.stride(-1) == 1 and d == k.get_device()
            and (frequencies is None or frequencies.dtype is torch.float32 and frequencies.dim() == 1
                 and frequencies.is_contiguous() and positions.dtype is torch.int32 and positions.shape == tokens
                 and positions.stride(-1) == 1 and frequencies.get_device() == d == positions.get_device())
            and (w is None or _is_weight(torch, w, w.dtype, dim, d) and (w is k_weight or k_weight is None
                                                                         or _is_weight(torch, k_weight, w.dtype, dim, d)))
            and (q_out is None or q_out.dtype is t and q_out.shape == shape and q_out.stride(-1) == 1 and q_out.get_device() == d)
            and (k_out is None or k_out.dtype is t and k_out.shape == rows and k_out.stride(-1) == 1 and k_out.get_device() == d)
        ):
            dev = d
    except (AttributeError, IndexError, RuntimeError, TypeError, ValueError):
        pass
    if dev < 0:
        _check_norm_rotate(q, k, positions, frequencies, q_weight, k_weight, (q_out, k_out))
        shape, rows = q.shape, k.shape
        w = k_weight if q_weight is None else q_weight
    if out is not None:
        _refuse_followed(q, k, frequencies, q_weight, k_weight, q_out, k_out)
    if q_out is None:
        q_out = q.new_empty(shape)
    if k_out is None:
        k_out = k.new_empty(rows)
    code = _dt_code(q.dtype)
    if len(shape) == 4:
        batch, tokens, heads, dim = shape
        steps = (*q.stride()[:3], *k.stride()[:3], *q_out.stride()[:3], *k_out.stride()[:3],
                 0 if frequencies is None else positions.stride(0))
    else:
        batch, (tokens, heads, dim) = 1, shape
        steps = (0, *q.stride()[:2], 0, *k.stride()[:2], 0, *q_out.stride()[:2], 0, *k_out.stride()[:2], 0)
    angles = (0, 0, 0) if frequencies is None else (2 * frequencies.shape[0], positions.data_ptr(), frequencies.data_ptr())
    a = _lib.NormRotateArgs()
    _pack(
        _ROTATE, a, code, code if w is None else _dt_code(w.dtype), batch, tokens, heads, rows[-2], dim, angles[0],
        bool(interleaved), eps is not None, 0.0 if eps is None else eps, q.data_ptr(), k.data_ptr(),
        0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(), angles[1], angles[2],
        q_out.data_ptr(), k_out.data_ptr(), *steps)
    _run(q, load().tf_exl3_norm_rotate, a)
    if out is not None:
        _changed(q_out, k_out)
    if _followed(q, k, frequencies, q_weight, k_weight):
        return tuple(_without_gradient("norm_rotate", o, x, frequencies, y)
                     for o, x, y in ((q_out, q, q_weight), (k_out, k, k_weight)))
    return q_out, k_out


# ---------------------------------------------------------------- whole prompts


def _check_prompt_attention(q, k, v, offsets, out):
    torch = _torch()
    _need("q", q, 3, _halves())
    tokens, heads, dim = q.shape
    same = (q.dtype,)
    _need("k", k, 3, same, (tokens, None, dim))
    _need("v", v, 3, same, tuple(k.shape))
    _need("offsets", offsets, 1, (torch.int32,))
    if offsets.shape[0] < 1:
        raise ValueError("offsets must have the sequences' beginnings and the last one's end")
    if out is not None:
        _need("out", out, 3, same, tuple(q.shape))
    _one_gpu(q, k, v, offsets, out)


def prompt_attention(q, k, v, offsets, scale=None, out=None):
    """out[tokens][q_heads][dim]: causal attention of prompts packed behind one another
    (tf_exl3_prompt_attention).

    q [tokens][q_heads][dim], k and v [tokens][kv_heads][dim] of fp16 or bf16 (views of a fused
    projection's rows will do); offsets int32 [batch + 1]: sequence b has the tokens offsets[b] ..
    offsets[b + 1] - 1, and each sees those of its sequence up to itself. Rows outside of all
    sequences are left as they are in `out` (without one: not set; refused where autograd follows a
    tensor). scale defaults to dim ** -0.5. How long the sequences are is not looked at on the host, so a captured call
    can be replayed with other offsets."""
    torch = _torch()
    dev = -1
    try:
        tokens, heads, dim = shape = q.shape
        rows, t, d = k.shape, q.dtype, q.get_device()
        if (
            (t is torch.bfloat16 or t is torch.float16) and k.dtype is t and v.dtype is t
            and rows == (tokens, rows[1], dim) and v.shape == rows
            and offsets.dtype is torch.int32 and len(offsets.shape) == 1 and offsets.shape[0] > 0 and offsets.stride(0) == 1
            and q.stride(2) == k.stride(2) == v.stride(2) == 1
            and d == k.get_device() == v.get_device() == offsets.get_device()
            and (out is None or out.dtype is t and out.shape == shape and out.stride(2) == 1 and out.get_device() == d)
        ):
            dev = d
    except (AttributeError, IndexError, RuntimeError, TypeError, ValueError):
        pass
    if dev < 0:
        _check_prompt_attention(q, k, v, offsets, out)
        tokens, heads, dim = shape = q.shape
        rows = k.shape
    given = out is not None
    if given:
        _refuse_followed(q, k, v, out)
    else:
        out = q.new_empty(shape)
    a = _lib.PromptAttentionArgs()
    _pack(
        _PROMPT, a, _dt_code(q.dtype), tokens, offsets.shape[0] - 1, heads, rows[1], dim,
        dim ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), offsets.data_ptr(), out.data_ptr(),
        *q.stride()[:2], *k.stride()[:2], *v.stride()[:2], *out.stride()[:2])
    _run(q, load().tf_exl3_prompt_attention, a)
    if given:
        _changed(out)
    if _followed(q, k, v):
        return _without_gradient("prompt_attention", out, q, k, v)
    return out


# ---------------------------------------------------------------- the cache in 4 bits


def _check_cache(k_cache, v_cache, table, lengths, batch, heads, dim):
    torch = _torch()
    _need("k_cache", k_cache, 4, (torch.uint8,), (None, None, heads, None if dim is None else q4_row_bytes(dim)))
    _need("v_cache", v_cache, 4, (torch.uint8,), tuple(k_cache.shape))
    if k_cache.shape[0] < 1 or k_cache.shape[1] < 1:
        raise ValueError("the cache must have at least one page of one slot")
    if k_cache.shape[3] < 20 or k_cache.shape[3] % 20:
        raise ValueError(f"rows of the cache must have q4_row_bytes(dim) bytes, not {k_cache.shape[3]}")
    _need("table", table, 2, (torch.int32,), (batch, None))
    _need("lengths", lengths, 1, (torch.int32,), (batch,))


def _cache_fits(torch, k_cache, v_cache, table, lengths, batch, heads, row, d):
    """Whether the arguments that every call with such a cache has pass their checks."""
    pages = k_cache.shape
    return (
        k_cache.dtype is torch.uint8 and v_cache.dtype is torch.uint8 and len(pages) == 4 and v_cache.shape == pages
        and pages[2] == heads and pages[3] == row and pages[0] > 0 and pages[1] > 0
        and k_cache.stride(3) == v_cache.stride(3) == 1
        and table.dtype is torch.int32 and len(table.shape) == 2 and table.shape[0] == batch and table.stride(1) == 1
        and lengths.dtype is torch.int32 and lengths.shape == (batch,) and lengths.stride(0) == 1
        and d >= 0 and d == k_cache.get_device() == v_cache.get_device() == table.get_device() == lengths.get_device()
    )


def _check_cache_append_q4(k, v, k_cache, v_cache, table, lengths, nodes, counts):
    torch = _torch()
    _need("k", k, 4, _floats())
    batch, tokens, heads, dim = k.shape
    _need("v", v, 4, (k.dtype,), (batch, tokens, heads, dim))
    _check_cache(k_cache, v_cache, table, lengths, batch, heads, dim)
    if nodes is not None:
        _need("nodes", nodes, 2, (torch.int32,), (batch, tokens))
        _whole("nodes", nodes)
    if counts is not None:
        _need("counts", counts, 1, (torch.int32,), (batch,))
    _one_gpu(k, v, k_cache, v_cache, table, lengths, nodes, counts)


def cache_append_q4(k, v, k_cache, v_cache, table, lengths, nodes=None, counts=None):
    """Writes rows of k and v [batch][tokens][kv_heads][dim] (fp32, fp16 or bf16) behind the
    lengths[b] positions that a sequence has in a cache in 4 bits (tf_exl3_cache_append_q4).
    k_cache, v_cache uint8 [pages][page_size][kv_heads][q4_row_bytes(dim)], in any order of memory
    with contiguous rows (a head's slots behind one another read fastest); the rest as in
    cache_append."""
    torch = _torch()
    fit = False
    try:
        batch, tokens, heads, dim = k.shape
        t, d = k.dtype, k.get_device()
        fit = (
            (t is torch.bfloat16 or t is torch.float16 or t is torch.float32) and v.dtype is t and v.shape == k.shape
            and k.stride(3) == v.stride(3) == 1 and v.get_device() == d and dim % 32 == 0
            and _cache_fits(torch, k_cache, v_cache, table, lengths, batch, heads, dim // 8 * 5, d)
            and (nodes is None or nodes.dtype is torch.int32 and nodes.shape == (batch, tokens) and nodes.is_contiguous()
                 and nodes.get_device() == d)
            and (counts is None or counts.dtype is torch.int32 and counts.shape == (batch,) and counts.stride(0) == 1
                 and counts.get_device() == d)
        )
    except (AttributeError, IndexError, RuntimeError, TypeError, ValueError):
        pass
    if not fit:
        _check_cache_append_q4(k, v, k_cache, v_cache, table, lengths, nodes, counts)
        batch, tokens, heads, dim = k.shape
    a = _lib.CacheAppendQ4Args()
    _pack(
        _APPEND, a, _dt_code(k.dtype), batch, tokens, heads, dim, *k_cache.shape[:2], table.shape[1], k.data_ptr(),
        v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), _ptr(nodes) or 0,
        _ptr(counts) or 0, *k.stride()[:3], *v.stride()[:3], *k_cache.stride()[:3], *v_cache.stride()[:3], table.stride(0))
    _run(k, load().tf_exl3_cache_append_q4, a)
    _changed(k_cache, v_cache)


def cache_read_q4(k_cache, v_cache, table, lengths, tokens, first=None, dtype=None):
    """(k, v) [batch][tokens][kv_heads][dim] of dtype (bf16 unless given): what positions first[b] + j of
    a cache in 4 bits stand for, from 0 where first int32 [batch] is None (tf_exl3_cache_read_q4).
    Rows from lengths[b] on are zeros."""
    torch = _torch()
    t = torch.bfloat16 if dtype is None else dtype
    if t not in _floats():
        raise ValueError(f"dtype must be {' or '.join(map(str, _floats()))}, not {t}")
    if not isinstance(tokens, int) or tokens < 0:
        raise ValueError(f"tokens must be a number of positions, not {tokens}")
    fit = False
    try:
        batch = table.shape[0]
        heads, row = k_cache.shape[2:]
        d = k_cache.get_device()
        fit = (
            row > 0 and row % 20 == 0 and _cache_fits(torch, k_cache, v_cache, table, lengths, batch, heads, row, d)
            and (first is None or first.dtype is torch.int32 and first.shape == (batch,) and first.stride(0) == 1
                 and first.get_device() == d)
        )
    except (AttributeError, IndexError, RuntimeError, TypeError, ValueError):
        pass
    if not fit:
        _need("table", table, 2, (torch.int32,))
        batch = table.shape[0]
        _check_cache(k_cache, v_cache, table, lengths, batch, None, None)
        if first is not None:
            _need("first", first, 1, (torch.int32,), (batch,))
        _one_gpu(k_cache, v_cache, table, lengths, first)
        heads, row = k_cache.shape[2:]
    dim = row * 8 // 5
    k, v = (torch.empty((batch, tokens, heads, dim), dtype=t, device=k_cache.device) for _ in range(2))
    a = _lib.CacheReadQ4Args()
    _pack(
        _READ, a, _dt_code(t), batch, tokens, heads, dim, *k_cache.shape[:2], table.shape[1], k_cache.data_ptr(),
        v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), _ptr(first) or 0, k.data_ptr(), v.data_ptr(),
        *k_cache.stride()[:3], *v_cache.stride()[:3], *k.stride()[:3], *v.stride()[:3], table.stride(0))
    _run(k_cache, load().tf_exl3_cache_read_q4, a)
    return k, v


def _check_tree_attention_q4(q, k, v, mask, k_cache, v_cache, table, lengths, out):
    torch = _torch()
    _need("q", q, 4, _halves())
    batch, nodes, hq, dim = q.shape
    same = (q.dtype,)
    _need("k", k, 4, same, (batch, nodes, None, dim))
    hkv = k.shape[2]
    _need("v", v, 4, same, (batch, nodes, hkv, dim))
    _need("mask", mask, 2, (torch.int64,), (batch, nodes))
    _whole("mask", mask)
    _check_cache(k_cache, v_cache, table, lengths, batch, hkv, dim)
    if out is not None:
        _need("out", out, 4, same, (batch, nodes, hq, dim))
    _one_gpu(q, k, v, mask, k_cache, v_cache, table, lengths, out)


def tree_attention_q4(q, k, v, mask, k_cache, v_cache, table, lengths, scale=None, out=None):
    """tree_attention over a cache in 4 bits (tf_exl3_tree_attention_q4): k_cache, v_cache uint8
    [pages][page_size][kv_heads][q4_row_bytes(dim)] as in cache_append_q4, everything else as
    in tree_attention, but that `out` is refused where autograd follows a tensor. A cached row is what
    cache_read_q4 gives in q's type."""
    torch = _torch()
    fit = False
    try:
        batch, nodes, hq, dim = shape = q.shape
        rows, t, d = k.shape, q.dtype, q.get_device()
        hkv = rows[2]
        fit = (
            (t is torch.bfloat16 or t is torch.float16) and k.dtype is t and v.dtype is t
            and rows == (batch, nodes, hkv, dim) and v.shape == rows and dim % 32 == 0
            and mask.dtype is torch.int64 and mask.shape == (batch, nodes) and mask.is_contiguous()
            and q.stride(3) == k.stride(3) == v.stride(3) == 1
            and d == k.get_device() == v.get_device() == mask.get_device()
            and _cache_fits(torch, k_cache, v_cache, table, lengths, batch, hkv, dim // 8 * 5, d)
            and (out is None or out.dtype is t and out.shape == shape and out.stride(3) == 1 and out.get_device() == d)
        )
    except (AttributeError, IndexError, RuntimeError, TypeError, ValueError):
        pass
    if not fit:
        _check_tree_attention_q4(q, k, v, mask, k_cache, v_cache, table, lengths, out)
        batch, nodes, hq, dim = shape = q.shape
        hkv = k.shape[2]
    given = out is not None
    if given:
        _refuse_followed(q, k, v, out)
    else:
        out = q.new_empty(shape)
    lib = load()
    pages, columns = k_cache.shape, table.shape[1]
    a = _lib.TreeAttentionArgs(_dt_code(q.dtype), batch, nodes, hq, hkv, dim, pages[0], pages[1], columns)
    need = lib.tf_exl3_tree_attention_q4_workspace(a)
    ws = _workspace(need, q)
    _pack(
        _ATTENTION, a, a.dtype, batch, nodes, hq, hkv, dim, pages[0], pages[1], columns,
        dim ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), mask.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), out.data_ptr(), ws.data_ptr(), need,
        *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *k_cache.stride()[:3], *v_cache.stride()[:3], *out.stride()[:3],
        table.stride(0))
    _run(q, lib.tf_exl3_tree_attention_q4, a)
    if given:
        _changed(out)
    if _followed(q, k, v):
        return _without_gradient("tree_attention_q4", out, q, k, v)
    return out
