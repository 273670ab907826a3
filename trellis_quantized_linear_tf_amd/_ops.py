"""The operators around the projection: attention of a tree of drafted tokens over a
paged cache, the cache's append, the verification of the drafts against the head's
logits, and the distillation that trains a drafter on a teacher's top logits.

Marshalling only, as in _lib: every argument is checked here (element types, shapes,
strides, one GPU), outputs and the workspace come from torch's allocator on the
current stream, and the library's kernels do the rest on that stream. The formulas,
and what happens to out-of-range values on the device, stand in include/tf_exl3.h.
"""

from __future__ import annotations

import functools
import struct

from . import _lib
from ._lib import _dt_code, _run, _torch, load


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


def _followed(*tensors) -> bool:
    """Whether autograd follows a tensor, backward or (a tangent within a dual level) forward."""
    torch = _torch()
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return True
    forward = torch.autograd.forward_ad
    return forward._current_level >= 0 and any(
        t is not None and forward.unpack_dual(t).tangent is not None for t in tensors)


def _refuse_followed(*tensors) -> None:
    """For tensors that a call with out= may not have in autograd's graph: what it writes there is in no graph, and a graph
    that goes through what was there before would not know of it."""
    if _followed(*tensors):
        raise ValueError(
            "out cannot be given here where autograd follows a tensor: call it without out, under torch.no_grad() or on "
            "detached tensors")


def _changed(*tensors) -> None:
    """Raises the versions of tensors that a call has written into: a backward pass that needs what was there fails."""
    _torch().autograd.graph.increment_version(tensors)


@functools.cache
def _nodes():
    """The calls' nodes in autograd's graph. None has a forward mode, which autograd itself refuses then."""
    torch = _torch()
    from torch.autograd.function import once_differentiable

    class WithoutGradient(torch.autograd.Function):
        """A result whose inputs it gives no gradient: asking for one is an error, not a zero."""

        @staticmethod
        def forward(ctx, name, result, *inputs):
            ctx.name = name
            return result.detach()

        @staticmethod
        def backward(ctx, *_):
            raise RuntimeError(f"{ctx.name} has no gradient: call it under torch.no_grad() or on detached tensors")

    class DistillLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, index, top, weight, temperature, want_grad):
            ctx.set_materialize_grads(False)  # a gradient's gradient would be as large as the logits
            ctx.save_for_backward(logits, index, top)
            ctx.temperature = temperature
            loss, grad = _distill(logits, index, top, weight, temperature, True, want_grad)
            if want_grad:
                ctx.mark_non_differentiable(grad)
            return loss, grad

        @staticmethod
        @once_differentiable
        def backward(ctx, weight, _):
            if weight is None:
                return (None,) * 6
            if ctx.needs_input_grad[2]:
                raise RuntimeError("the distillation loss has no gradient by the teacher's logits: pass top.detach()")
            logits, index, top = ctx.saved_tensors
            grad = _distill(logits, index, top, weight.contiguous(), ctx.temperature, False, True)[1]
            return grad, None, None, None, None, None

    return WithoutGradient, DistillLoss


# Every call looks its arguments over with one chain of comparisons, which implies all of
# the checks below and costs a few microseconds; only a call that does not pass it goes
# through them one by one, for the message (or because a dimension of 1 has an odd stride).
_ATTENTION = struct.Struct("@9if10QN19q")
_APPEND = struct.Struct("@8i8Q13q")


def _pack(layout, args, *values):
    try:
        layout.pack_into(args, 0, *values)
    except (OverflowError, struct.error):
        raise ValueError("a size or stride is out of the library's range") from None


def _sizes(*sizes):
    """Numbers that the library takes as 32-bit integers."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"sizes must be below 2^31, not {max(sizes)}")


def _check_cache(k_cache, v_cache, table, lengths, dtypes, batch, heads, dim):
    torch = _torch()
    _need("k_cache", k_cache, 4, dtypes, (None, None, heads, dim))
    _need("v_cache", v_cache, 4, dtypes, tuple(k_cache.shape))
    if k_cache.shape[0] < 1 or k_cache.shape[1] < 1:
        raise ValueError("the cache must have at least one page of one slot")
    _need("table", table, 2, (torch.int32,), (batch, None))
    _need("lengths", lengths, 1, (torch.int32,), (batch,))


def _check_tree_attention(q, k, v, mask, k_cache, v_cache, table, lengths, out):
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


def tree_attention(q, k, v, mask, k_cache, v_cache, table, lengths, scale=None, out=None):
    """out[batch][nodes][q_heads][dim]: attention of drafted nodes over their sequence's cache
    and, by a mask, over each other (tf_exl3_tree_attention).

    q [batch][nodes][q_heads][dim], k and v [batch][nodes][kv_heads][dim] of fp16 or bf16: the
    nodes' own rows (views of a fused projection's rows will do). mask int64 [batch][nodes]:
    bit t of a node's mask says that it sees node t (1..64 nodes). k_cache, v_cache [pages]
    [page_size][kv_heads][dim], in any order of memory with contiguous rows; table int32
    [batch][table_pages]; lengths int32 [batch]: positions in the cache, all of them seen.
    scale defaults to dim ** -0.5. A node that sees nothing gets zeros.

    It has no gradient: where autograd follows an input, the result (not `out` itself) is part of
    its graph, and a backward pass that reaches it raises. An `out` that autograd follows is refused."""
    torch = _torch()
    dev = -1
    try:
        batch, nodes, hq, dim = shape = q.shape
        rows, pages = k.shape, k_cache.shape
        hkv, columns, t = rows[2], table.shape[1], q.dtype
        sq, sk, sv, skc, svc = q.stride(), k.stride(), v.stride(), k_cache.stride(), v_cache.stride()
        if (
            (t is torch.bfloat16 or t is torch.float16)
            and k.dtype is t and v.dtype is t and k_cache.dtype is t and v_cache.dtype is t
            and rows == (batch, nodes, hkv, dim) and v.shape == rows
            and len(pages) == 4 and pages[2] == hkv and pages[3] == dim and pages[0] > 0 and pages[1] > 0
            and v_cache.shape == pages
            and mask.dtype is torch.int64 and mask.shape == (batch, nodes) and mask.is_contiguous()
            and table.dtype is torch.int32 and table.shape == (batch, columns) and table.stride(1) == 1
            and lengths.dtype is torch.int32 and lengths.shape == (batch,) and lengths.stride(0) == 1
            and sq[3] == sk[3] == sv[3] == skc[3] == svc[3] == 1
            and (out is None or out.dtype is t and out.shape == shape and out.stride(3) == 1)
        ):
            d = q.get_device()
            if (
                d == k.get_device() == v.get_device() == mask.get_device() == k_cache.get_device()
                == v_cache.get_device() == table.get_device() == lengths.get_device()
                and (out is None or out.get_device() == d)
            ):
                dev = d
    except (AttributeError, IndexError, RuntimeError, ValueError):
        pass
    if dev < 0:
        _check_tree_attention(q, k, v, mask, k_cache, v_cache, table, lengths, out)
    given = out is not None
    if given:
        _refuse_followed(out)
    else:
        out = q.new_empty(shape)
    lib = load()
    a = _lib.TreeAttentionArgs(_dt_code(t), batch, nodes, hq, hkv, dim, pages[0], pages[1], columns)
    need = lib.tf_exl3_tree_attention_workspace(a)
    ws = _workspace(need, q)
    _pack(
        _ATTENTION, a, a.dtype, batch, nodes, hq, hkv, dim, pages[0], pages[1], columns,
        dim ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), mask.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), out.data_ptr(), ws.data_ptr(), need,
        *sq[:3], *sk[:3], *sv[:3], *skc[:3], *svc[:3], *out.stride()[:3], table.stride(0))
    _run(q, lib.tf_exl3_tree_attention, a)
    if given:
        _changed(out)
    if _followed(q, k, v, k_cache, v_cache):
        return _nodes()[0].apply("tree_attention", out, q, k, v, k_cache, v_cache)
    return out


def _check_cache_append(k, v, k_cache, v_cache, table, lengths, nodes, counts):
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


def cache_append(k, v, k_cache, v_cache, table, lengths, nodes=None, counts=None):
    """Writes rows of k and v [batch][tokens][kv_heads][dim] behind the lengths[b] positions
    that a sequence has in the cache (tf_exl3_cache_append). nodes int32 [batch][tokens] and
    counts int32 [batch] choose them: position lengths[b] + j takes row nodes[b][j], for
    j < counts[b] (verify_tree's `accepted` and `count` fit). lengths stays as it is. The cache
    takes values: to autograd its rows are constants."""
    torch = _torch()
    dev = -1
    try:
        batch, tokens, heads, dim = rows = k.shape
        pages, columns, t = k_cache.shape, table.shape[1], k.dtype
        sk, sv, skc, svc = k.stride(), v.stride(), k_cache.stride(), v_cache.stride()
        if (
            (t is torch.bfloat16 or t is torch.float16)
            and v.dtype is t and k_cache.dtype is t and v_cache.dtype is t and v.shape == rows
            and len(pages) == 4 and pages[2] == heads and pages[3] == dim and pages[0] > 0 and pages[1] > 0
            and v_cache.shape == pages
            and table.dtype is torch.int32 and table.shape == (batch, columns) and table.stride(1) == 1
            and lengths.dtype is torch.int32 and lengths.shape == (batch,) and lengths.stride(0) == 1
            and sk[3] == sv[3] == skc[3] == svc[3] == 1
            and (nodes is None or nodes.dtype is torch.int32 and nodes.shape == (batch, tokens) and nodes.is_contiguous())
            and (counts is None or counts.dtype is torch.int32 and counts.shape == (batch,) and counts.stride(0) == 1)
        ):
            d = k.get_device()
            if (
                d == v.get_device() == k_cache.get_device() == v_cache.get_device() == table.get_device()
                == lengths.get_device()
                and (nodes is None or nodes.get_device() == d) and (counts is None or counts.get_device() == d)
            ):
                dev = d
    except (AttributeError, IndexError, RuntimeError, ValueError):
        pass
    if dev < 0:
        _check_cache_append(k, v, k_cache, v_cache, table, lengths, nodes, counts)
    a = _lib.CacheAppendArgs()
    _pack(
        _APPEND, a, k.element_size(), batch, tokens, heads, dim, pages[0], pages[1], columns, k.data_ptr(), v.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), _ptr(nodes) or 0, _ptr(counts) or 0,
        *sk[:3], *sv[:3], *skc[:3], *svc[:3], table.stride(0))
    _run(k, load().tf_exl3_cache_append, a)
    _changed(k_cache, v_cache)


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


def _drafts_fit(torch, logits, tokens, u, temperature):
    """Whether the arguments that both verifications have pass their checks, and (batch, nodes, vocab)."""
    sizes = batch, nodes, vocab = logits.shape
    t, d, pairs = logits.dtype, logits.get_device(), (batch, nodes)
    return (
        (t is torch.float32 or t is torch.bfloat16 or t is torch.float16) and logits.stride(2) == 1
        and tokens.dtype is torch.int32 and tokens.shape == pairs and tokens.is_contiguous()
        and u.dtype is torch.float32 and u.shape == pairs and u.is_contiguous()
        and d == tokens.get_device() == u.get_device() and d >= 0
        and (temperature is None or temperature.dtype is torch.float32 and temperature.shape == (batch,)
             and temperature.stride(0) == 1 and temperature.get_device() == d)
    ), sizes


def verify_tree(logits, tokens, parents, u, temperature=None):
    """(accepted int32 [batch][nodes], count int32 [batch], next int32 [batch]): the path of a
    drafted tree that the target's own samples follow (tf_exl3_verify_tree).

    logits [batch][nodes][vocab] of the target at every node (fp32, fp16 or bf16); tokens and
    parents int32 [batch][nodes], node 0 the last token before the drafts; u fp32 [batch]
    [nodes]: a random number in [0, 1) for each row; temperature fp32 [batch], 0 for the
    largest logit, None for 1. accepted holds the path's nodes, then -1; next the token
    sampled at its end."""
    torch = _torch()
    fit = False
    try:
        drafts, (batch, nodes, vocab) = _drafts_fit(torch, logits, tokens, u, temperature)
        fit = drafts and (parents.dtype is torch.int32 and parents.shape == (batch, nodes) and parents.is_contiguous()
                          and parents.get_device() == logits.get_device())
    except (AttributeError, IndexError, RuntimeError, ValueError):
        pass
    if not fit:
        batch, nodes, vocab = _check_drafts(logits, tokens, u, temperature)
        _need("parents", parents, 2, (torch.int32,), (batch, nodes))
        _whole("parents", parents)
        _one_gpu(logits, tokens, parents, u, temperature)
    _sizes(batch, nodes, vocab)
    accepted = tokens.new_empty((batch, nodes))
    count, after = tokens.new_empty((batch,)), tokens.new_empty((batch,))
    lib = load()
    need = lib.tf_exl3_verify_workspace(batch, nodes, vocab)
    ws = _workspace(need, logits)
    _run(logits, lib.tf_exl3_verify_tree,
        _dt_code(logits.dtype), batch, nodes, vocab, logits.data_ptr(), logits.stride(0), logits.stride(1),
        tokens.data_ptr(), parents.data_ptr(), u.data_ptr(), _ptr(temperature), accepted.data_ptr(),
        count.data_ptr(), after.data_ptr(), ws.data_ptr(), ws.numel())
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
    fit = False
    try:
        drafts, (batch, nodes, vocab) = _drafts_fit(torch, logits, tokens, u, temperature)
        fit = drafts and (q.dtype is torch.float32 and q.shape == (batch, nodes - 1, vocab) and q.stride(2) == 1
                          and q.get_device() == logits.get_device())
    except (AttributeError, IndexError, RuntimeError, ValueError):
        pass
    if not fit:
        batch, nodes, vocab = _check_drafts(logits, tokens, u, temperature)
        _need("q", q, 3, (torch.float32,), (batch, max(nodes - 1, 0), vocab))
        _one_gpu(logits, tokens, q, u, temperature)
    _sizes(batch, nodes, vocab)
    count, after = tokens.new_empty((batch,)), tokens.new_empty((batch,))
    lib = load()
    need = lib.tf_exl3_verify_workspace(batch, nodes, vocab)
    ws = _workspace(need, logits)
    _run(logits, lib.tf_exl3_verify_chain,
        _dt_code(logits.dtype), batch, nodes, vocab, logits.data_ptr(), logits.stride(0), logits.stride(1),
        tokens.data_ptr(), _ptr(q) if nodes > 1 else None, q.stride(0), q.stride(1), u.data_ptr(),
        _ptr(temperature), count.data_ptr(), after.data_ptr(), ws.data_ptr(), ws.numel())
    return count, after


def _distill(logits, index, top, weight, temperature, want_loss, want_grad):
    torch = _torch()
    fit = False
    try:
        rows, vocab = logits.shape
        t, y, d, entries = logits.dtype, top.dtype, logits.get_device(), index.shape
        fit = (
            (t is torch.float32 or t is torch.bfloat16 or t is torch.float16) and logits.stride(1) == 1
            and (y is t or y is torch.float32 or y is torch.bfloat16 or y is torch.float16)
            and index.dtype is torch.int32 and len(entries) == 2 and entries[0] == rows and index.is_contiguous()
            and top.shape == entries and top.is_contiguous() and d == index.get_device() == top.get_device() and d >= 0
            and (weight is None and not want_grad or weight.dtype is torch.float32 and weight.shape == (rows,)
                 and weight.is_contiguous() and weight.get_device() == d)
        )
    except (AttributeError, IndexError, RuntimeError, ValueError):
        pass
    if not fit:
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
    _sizes(rows, vocab, index.shape[1])
    loss = torch.empty((rows,), dtype=torch.float32, device=logits.device) if want_loss else None
    grad = logits.new_empty((rows, vocab)) if want_grad else None
    lib = load()
    code = _dt_code(logits.dtype)
    need = lib.tf_exl3_distill_workspace(code, rows, vocab, index.shape[1])
    ws = _workspace(need, logits)
    _run(logits, lib.tf_exl3_distill,
        code, rows, vocab, index.shape[1], logits.data_ptr(), logits.stride(0), index.data_ptr(), top.data_ptr(),
        _dt_code(top.dtype), _ptr(weight), temperature, _ptr(loss), _ptr(grad), vocab, ws.data_ptr(), ws.numel())
    return loss, grad


def distill_loss(logits, index, top, temperature=1.0):
    """loss fp32 [rows] of logits [rows][vocab] against a teacher's top logits: top [rows]
    [top_k] at the places index int32 [rows][top_k], entries with an index outside the
    vocabulary (-1) left out (tf_exl3_distill). Under autograd its backward pass is distill_grad;
    there is none by the teacher's logits, and no second one."""
    if _followed(logits, top):
        return _nodes()[1].apply(logits, index, top, None, temperature, False)[0]
    return _distill(logits, index, top, None, temperature, True, False)[0]


def distill_grad(logits, index, top, weight, temperature=1.0):
    """The gradient of sum(weight * loss) by logits, of the logits' type; weight fp32 [rows]. To
    autograd it is a constant."""
    return _distill(logits, index, top, weight, temperature, False, True)[1]


def distill(logits, index, top, weight, temperature=1.0):
    """(loss, grad) in one call: distill_loss, which autograd may follow, and distill_grad."""
    if _followed(logits, top):
        return _nodes()[1].apply(logits, index, top, weight, temperature, True)
    return _distill(logits, index, top, weight, temperature, True, True)
