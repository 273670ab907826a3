"""The operators around the projection: attention of a tree of drafted tokens over a
paged cache, the cache's append, the verification of the drafts against the head's
logits, and the distillation that trains a drafter on a teacher's top logits.

Marshalling only, as in _lib: every argument is checked here (element types, shapes,
strides, one GPU), outputs and the workspace come from torch's allocator on the
current stream, and the library's kernels do the rest on that stream. The formulas,
and what happens to out-of-range values on the device, stand in include/tf_exl3.h.
"""

from __future__ import annotations

import ctypes

from . import _lib
from ._lib import _check, _dt_code, _stream, _torch, load


def _need(name, t, dim, dtypes, shape=None):
    """Element type, rank and shape of a tensor (None in shape: any size); contiguous innermost."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have element type {' or '.join(map(str, dtypes))}, not {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, not {t.dim()}")
    if shape is not None and any(w is not None and w != n for w, n in zip(shape, t.shape)):
        want = ", ".join("any" if w is None else str(w) for w in shape)
        raise ValueError(f"{name} must have shape ({want}), not {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _whole(name, t):
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _one_gpu(*tensors):
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        d = t.get_device()
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError("all tensors must be on one GPU")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(nbytes, like):
    """Device memory for one call; freed in stream order, so it may go out of scope at once."""
    torch = _torch()
    return torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=like.device)


def _halves():
    torch = _torch()
    return (torch.float16, torch.bfloat16)


def _floats():
    torch = _torch()
    return (torch.float32, torch.float16, torch.bfloat16)


_L3 = ctypes.c_int64 * 3


def _strides(t):
    return _L3(*(s if n > 1 else 0 for s, n in zip(t.stride()[:3], t.shape)))  # a dimension of 1 has any stride


def _check_cache(k_cache, v_cache, table, lengths, dtypes, batch, heads, dim):
    torch = _torch()
    _need("k_cache", k_cache, 4, dtypes, (None, None, heads, dim))
    _need("v_cache", v_cache, 4, dtypes, tuple(k_cache.shape))
    if k_cache.shape[0] < 1 or k_cache.shape[1] < 1:
        raise ValueError("the cache must have at least one page of one slot")
    _need("table", table, 2, (torch.int32,), (batch, None))
    _need("lengths", lengths, 1, (torch.int32,), (batch,))


def tree_attention(q, k, v, mask, k_cache, v_cache, table, lengths, scale=None, out=None):
    """out[batch][nodes][q_heads][dim]: attention of drafted nodes over their sequence's cache
    and, by a mask, over each other (tf_exl3_tree_attention).

    q [batch][nodes][q_heads][dim], k and v [batch][nodes][kv_heads][dim] of fp16 or bf16: the
    nodes' own rows (views of a fused projection's rows will do). mask int64 [batch][nodes]:
    bit t of a node's mask says that it sees node t (1..64 nodes). k_cache, v_cache [pages]
    [page_size][kv_heads][dim], in any order of memory with contiguous rows; table int32
    [batch][table_pages]; lengths int32 [batch]: positions in the cache, all of them seen.
    scale defaults to dim ** -0.5. A node that sees nothing gets zeros."""
    torch = _torch()
    _need("q", q, 4, _halves())
    batch, nodes, hq, dim = q.shape
    same = (q.dtype,)
    _need("k", k, 4, same, (batch, nodes, None, dim))
    hkv = k.shape[2]
    _need("v", v, 4, same, (batch, nodes, hkv, dim))
    _need("mask", mask, 2, (torch.int64,), (batch, nodes))
    _whole("mask", mask)
    _check_cache(k_cache, v_cache, table, lengths, same, batch, hkv, dim)
    if out is not None:
        _need("out", out, 4, same, (batch, nodes, hq, dim))
    _one_gpu(q, k, v, mask, k_cache, v_cache, table, lengths, out)
    if out is None:
        out = torch.empty((batch, nodes, hq, dim), dtype=q.dtype, device=q.device)
    a = _lib.TreeAttentionArgs(
        _dt_code(q.dtype), batch, nodes, hq, hkv, dim, k_cache.shape[0], k_cache.shape[1], table.shape[1],
        dim ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), mask.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), out.data_ptr())
    a.q_stride, a.k_stride, a.v_stride = _strides(q), _strides(k), _strides(v)
    a.k_cache_stride, a.v_cache_stride, a.out_stride = _strides(k_cache), _strides(v_cache), _strides(out)
    a.table_stride = table.stride(0)
    lib = load()
    a.workspace_bytes = lib.tf_exl3_tree_attention_workspace(a)
    ws = _workspace(a.workspace_bytes, q)
    a.workspace = ws.data_ptr()
    _check(lib.tf_exl3_tree_attention(a, _stream(q)))
    return out


def cache_append(k, v, k_cache, v_cache, table, lengths, nodes=None, counts=None):
    """Writes rows of k and v [batch][tokens][kv_heads][dim] behind the lengths[b] positions
    that a sequence has in the cache (tf_exl3_cache_append). nodes int32 [batch][tokens] and
    counts int32 [batch] choose them: position lengths[b] + j takes row nodes[b][j], for
    j < counts[b] (verify_tree's `accepted` and `count` fit). lengths stays as it is."""
    torch = _torch()
    dtypes = (torch.float16, torch.bfloat16, torch.float32, torch.int8, torch.uint8, torch.int16, torch.float8_e4m3fn,
              torch.float8_e5m2)
    _need("k", k, 4, dtypes)
    batch, tokens, heads, dim = k.shape
    same = (k.dtype,)
    _need("v", v, 4, same, (batch, tokens, heads, dim))
    _check_cache(k_cache, v_cache, table, lengths, same, batch, heads, dim)
    if nodes is not None:
        _need("nodes", nodes, 2, (torch.int32,), (batch, tokens))
        _whole("nodes", nodes)
    if counts is not None:
        _need("counts", counts, 1, (torch.int32,), (batch,))
    _one_gpu(k, v, k_cache, v_cache, table, lengths, nodes, counts)
    a = _lib.CacheAppendArgs(
        k.element_size(), batch, tokens, heads, dim, k_cache.shape[0], k_cache.shape[1], table.shape[1],
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        _ptr(nodes), _ptr(counts), _strides(k), _strides(v), _strides(k_cache), _strides(v_cache), table.stride(0))
    _check(load().tf_exl3_cache_append(a, _stream(k)))


def _check_drafts(logits, tokens, u, temperature):
    torch = _torch()
    _need("logits", logits, 3, _floats())
    batch, nodes, vocab = logits.shape
    _need("tokens", tokens, 2, (torch.int32,), (batch, nodes))
    _need("u", u, 2, (torch.float32,), (batch, nodes))
    if temperature is not None:
        _need("temperature", temperature, 1, (torch.float32,), (batch,))
    for name, t in (("tokens", tokens), ("u", u)):
        _whole(name, t)
    return batch, nodes, vocab


def verify_tree(logits, tokens, parents, u, temperature=None):
    """(accepted int32 [batch][nodes], count int32 [batch], next int32 [batch]): the path of a
    drafted tree that the target's own samples follow (tf_exl3_verify_tree).

    logits [batch][nodes][vocab] of the target at every node (fp32, fp16 or bf16); tokens and
    parents int32 [batch][nodes], node 0 the last token before the drafts; u fp32 [batch]
    [nodes]: a random number in [0, 1) for each row; temperature fp32 [batch], 0 for the
    largest logit, None for 1. accepted holds the path's nodes, then -1; next the token
    sampled at its end."""
    torch = _torch()
    batch, nodes, vocab = _check_drafts(logits, tokens, u, temperature)
    _need("parents", parents, 2, (torch.int32,), (batch, nodes))
    _whole("parents", parents)
    _one_gpu(logits, tokens, parents, u, temperature)
    accepted = torch.empty((batch, nodes), dtype=torch.int32, device=logits.device)
    count, after = torch.empty((2, batch), dtype=torch.int32, device=logits.device)
    lib = load()
    need = lib.tf_exl3_verify_workspace(batch, nodes, vocab)
    ws = _workspace(need, logits)
    _check(lib.tf_exl3_verify_tree(
        _dt_code(logits.dtype), batch, nodes, vocab, logits.data_ptr(), logits.stride(0), logits.stride(1),
        tokens.data_ptr(), parents.data_ptr(), u.data_ptr(), _ptr(temperature), accepted.data_ptr(),
        count.data_ptr(), after.data_ptr(), ws.data_ptr(), ws.numel(), _stream(logits)))
    return accepted, count, after


def verify_chain(logits, tokens, q, u, temperature=None):
    """(count int32 [batch], next int32 [batch]): speculative sampling of a drafted chain
    (tf_exl3_verify_chain).

    logits [batch][nodes][vocab] of the target; tokens int32 [batch][nodes], the last token
    and then the drafts; q fp32 [batch][nodes - 1][vocab]: the probabilities that each draft
    was drawn from; u fp32 [batch][nodes]: random numbers in [0, 1), one for each draft and
    the last for the token after them. count is 1 + the accepted drafts; next comes from
    max(p - q, 0) where a draft was refused, from p where all were accepted."""
    torch = _torch()
    batch, nodes, vocab = _check_drafts(logits, tokens, u, temperature)
    _need("q", q, 3, (torch.float32,), (batch, max(nodes - 1, 0), vocab))
    _one_gpu(logits, tokens, q, u, temperature)
    count, after = torch.empty((2, batch), dtype=torch.int32, device=logits.device)
    lib = load()
    need = lib.tf_exl3_verify_workspace(batch, nodes, vocab)
    ws = _workspace(need, logits)
    _check(lib.tf_exl3_verify_chain(
        _dt_code(logits.dtype), batch, nodes, vocab, logits.data_ptr(), logits.stride(0), logits.stride(1),
        tokens.data_ptr(), _ptr(q) if nodes > 1 else None, q.stride(0), q.stride(1), u.data_ptr(),
        _ptr(temperature), count.data_ptr(), after.data_ptr(), ws.data_ptr(), ws.numel(), _stream(logits)))
    return count, after


def _distill(logits, index, top, weight, temperature, want_loss, want_grad):
    torch = _torch()
    _need("logits", logits, 2, _floats())
    rows, vocab = logits.shape
    _need("index", index, 2, (torch.int32,), (rows, None))
    _need("top", top, 2, _floats(), tuple(index.shape))
    _whole("index", index)
    _whole("top", top)
    if want_grad:
        _need("weight", weight, 1, (torch.float32,), (rows,))
        _whole("weight", weight)
    _one_gpu(logits, index, top, weight)
    loss = torch.empty((rows,), dtype=torch.float32, device=logits.device) if want_loss else None
    grad = torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device) if want_grad else None
    lib = load()
    code = _dt_code(logits.dtype)
    need = lib.tf_exl3_distill_workspace(code, rows, vocab, index.shape[1])
    ws = _workspace(need, logits)
    _check(lib.tf_exl3_distill(
        code, rows, vocab, index.shape[1], logits.data_ptr(), logits.stride(0), index.data_ptr(), top.data_ptr(),
        _dt_code(top.dtype), _ptr(weight), temperature, _ptr(loss), _ptr(grad), vocab, ws.data_ptr(), ws.numel(),
        _stream(logits)))
    return loss, grad


def distill_loss(logits, index, top, temperature=1.0):
    """loss fp32 [rows] of logits [rows][vocab] against a teacher's top logits: top [rows]
    [top_k] at the places index int32 [rows][top_k], entries with an index outside the
    vocabulary (-1) left out (tf_exl3_distill)."""
    return _distill(logits, index, top, None, temperature, True, False)[0]


def distill_grad(logits, index, top, weight, temperature=1.0):
    """The gradient of sum(weight * loss) by logits, of the logits' type; weight fp32 [rows]."""
    return _distill(logits, index, top, weight, temperature, False, True)[1]


def distill(logits, index, top, weight, temperature=1.0):
    """(loss, grad) in one call: distill_loss and distill_grad."""
    return _distill(logits, index, top, weight, temperature, True, True)
