"""Refusals of the operators around the projection, on the host (no GPU): the binding's
argument checks, reached from CPU tensors, and the library's own, reached with pointers
that are never dereferenced. Nothing here launches a kernel."""

import ctypes

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from trellis_quantized_linear_tf_amd import _lib

B, N, HQ, HKV, D, PAGE = 2, 4, 4, 2, 64, 16
bf = torch.bfloat16


def attn(**kw):
    a = dict(q=torch.zeros(B, N, HQ, D, dtype=bf), k=torch.zeros(B, N, HKV, D, dtype=bf),
             v=torch.zeros(B, N, HKV, D, dtype=bf), mask=torch.zeros(B, N, dtype=torch.int64),
             k_cache=torch.zeros(5, PAGE, HKV, D, dtype=bf), v_cache=torch.zeros(5, PAGE, HKV, D, dtype=bf),
             table=torch.zeros(B, 2, dtype=torch.int32), lengths=torch.zeros(B, dtype=torch.int32))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,msg", [
    (dict(q=torch.zeros(B, N, HQ, D)), "q must have element type"),
    (dict(q=torch.zeros(B, HQ, D, dtype=bf)), "q must have 4 dimensions"),
    (dict(k=torch.zeros(B, N, HKV, D, dtype=torch.float16)), "k must have element type"),
    (dict(k=torch.zeros(B, N + 1, HKV, D, dtype=bf)), "k must have shape"),
    (dict(v=torch.zeros(B, N, HKV + 1, D, dtype=bf)), "v must have shape"),
    (dict(mask=torch.zeros(B, N, dtype=torch.int32)), "mask must have element type"),
    (dict(mask=torch.zeros(B, N, 2, dtype=torch.int64)[..., 0]), "mask must be contiguous"),
    (dict(k_cache=torch.zeros(5, PAGE, HKV + 1, D, dtype=bf)), "k_cache must have shape"),
    (dict(v_cache=torch.zeros(4, PAGE, HKV, D, dtype=bf)), "v_cache must have shape"),
    (dict(k_cache=torch.zeros(5, PAGE, D, HKV, dtype=bf).transpose(2, 3)), "contiguous in its last"),
    (dict(k_cache=torch.zeros(0, PAGE, HKV, D, dtype=bf), v_cache=torch.zeros(0, PAGE, HKV, D, dtype=bf)), "at least one page"),
    (dict(table=torch.zeros(B, 2, dtype=torch.int64)), "table must have element type"),
    (dict(table=torch.zeros(B + 1, 2, dtype=torch.int32)), "table must have shape"),
    (dict(lengths=torch.zeros(B + 1, dtype=torch.int32)), "lengths must have shape"),
    (dict(out=torch.zeros(B, N, HQ, D)), "out must have element type"),
    (dict(out=torch.zeros(B, N, HQ, 2 * D, dtype=bf)), "out must have shape"),
    (dict(), "on the GPU"),
])
def test_tree_attention_refusals(bad, msg):
    with pytest.raises(ValueError, match=msg):
        tq.tree_attention(**attn(**bad))


@pytest.mark.parametrize("bad,msg", [
    (dict(k=torch.zeros(B, N, HKV, D, dtype=torch.int64)), "k must have element type"),
    (dict(v=torch.zeros(B, N, HKV, D)), "v must have element type"),
    (dict(nodes=torch.zeros(B, N + 1, dtype=torch.int32)), "nodes must have shape"),
    (dict(nodes=torch.zeros(B, N, dtype=torch.int64)), "nodes must have element type"),
    (dict(counts=torch.zeros(B, 1, dtype=torch.int32)), "counts must have 1 dim"),
    (dict(k_cache=torch.zeros(5, PAGE, HKV, D // 2, dtype=bf)), "k_cache must have shape"),
    (dict(), "on the GPU"),
])
def test_cache_append_refusals(bad, msg):
    a = attn(**bad)
    with pytest.raises(ValueError, match=msg):
        tq.cache_append(a["k"], a["v"], a["k_cache"], a["v_cache"], a["table"], a["lengths"], a.get("nodes"),
                        a.get("counts"))


V = 100


def drafts(**kw):
    a = dict(logits=torch.zeros(B, N, V), tokens=torch.zeros(B, N, dtype=torch.int32),
             parents=torch.zeros(B, N, dtype=torch.int32), q=torch.zeros(B, N - 1, V), u=torch.zeros(B, N),
             temperature=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,msg", [
    (dict(logits=torch.zeros(B, N, V, dtype=torch.float64)), "logits must have element type"),
    (dict(logits=torch.zeros(N, V)), "logits must have 3"),
    (dict(logits=torch.zeros(B, N, 2 * V)[..., ::2]), "contiguous in its last"),
    (dict(tokens=torch.zeros(B, N, dtype=torch.int64)), "tokens must have element type"),
    (dict(tokens=torch.zeros(B, N + 1, dtype=torch.int32)), "tokens must have shape"),
    (dict(u=torch.zeros(B, N, dtype=torch.float64)), "u must have element type"),
    (dict(u=torch.zeros(N, B).t()), "u must be contiguous|contiguous in its last"),
    (dict(temperature=torch.zeros(N)), "temperature must have shape"),
    (dict(), "on the GPU"),
])
def test_verify_refusals(bad, msg):
    a = drafts(**bad)
    with pytest.raises(ValueError, match=msg):
        tq.verify_tree(a["logits"], a["tokens"], a["parents"], a["u"], a["temperature"])
    with pytest.raises(ValueError, match=msg):
        tq.verify_chain(a["logits"], a["tokens"], a["q"], a["u"], a["temperature"])


def test_verify_refuses_other_parents_and_drafters():
    a = drafts(parents=torch.zeros(B, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="parents must have shape"):
        tq.verify_tree(a["logits"], a["tokens"], a["parents"], a["u"])
    for q, msg in ((torch.zeros(B, N, V), "q must have shape"), (torch.zeros(B, N - 1, V, dtype=bf), "element type")):
        with pytest.raises(ValueError, match=msg):
            tq.verify_chain(a["logits"], a["tokens"], q, a["u"])


def rows(**kw):
    a = dict(logits=torch.zeros(3, V), index=torch.zeros(3, 5, dtype=torch.int32), top=torch.zeros(3, 5),
             weight=torch.zeros(3))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,msg", [
    (dict(logits=torch.zeros(V)), "logits must have 2"),
    (dict(logits=torch.zeros(3, V, dtype=torch.int32)), "logits must have element type"),
    (dict(index=torch.zeros(3, 5, dtype=torch.int64)), "index must have element type"),
    (dict(index=torch.zeros(2, 5, dtype=torch.int32)), "index must have shape"),
    (dict(top=torch.zeros(3, 4)), "top must have shape"),
    (dict(top=torch.zeros(3, 10)[:, :5]), "top must be contiguous"),
    (dict(weight=torch.zeros(4)), "weight must have shape"),
    (dict(weight=None), "weight is required"),
    (dict(), "on the GPU"),
])
def test_distill_refusals(bad, msg):
    a = rows(**bad)
    for call in (tq.distill, tq.distill_grad):
        with pytest.raises(ValueError, match=msg):
            call(a["logits"], a["index"], a["top"], a["weight"])
    if "weight" not in bad:
        with pytest.raises(ValueError, match=msg):
            tq.distill_loss(a["logits"], a["index"], a["top"])


# ---------------------------------------------------------------- the library's own refusals

FAKE = 0x7F0000000000  # never dereferenced
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not _lib.LIB_PATH.exists():
        from trellis_quantized_linear_tf_amd._build import build

        build()
    return _lib.load()


def attention_args(lib, **kw):
    a = _lib.TreeAttentionArgs(2, B, N, HQ, HKV, D, 5, PAGE, 2, 0.125)
    for i, name in enumerate(("q", "k", "v", "mask", "k_cache", "v_cache", "table", "lengths", "out", "workspace")):
        setattr(a, name, FAKE + i * 512 * MB)
    a.q_stride[:] = a.out_stride[:] = (N * HQ * D, HQ * D, D)
    a.k_stride[:] = a.v_stride[:] = (N * HKV * D, HKV * D, D)
    a.k_cache_stride[:] = a.v_cache_stride[:] = (PAGE * HKV * D, HKV * D, D)
    a.table_stride = 2
    a.workspace_bytes = lib.tf_exl3_tree_attention_workspace(a)
    for name, value in kw.items():
        if name.endswith("_stride") and name != "table_stride":
            getattr(a, name)[:] = value
        else:
            setattr(a, name, value)
    return a


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=0), -4), (dict(dtype=3), -4), (dict(batch=-1), -10), (dict(batch=65536), -10), (dict(nodes=0), -10),
    (dict(nodes=65), -10), (dict(kv_heads=3), -10), (dict(kv_heads=0), -10), (dict(head_dim=72), -10),
    (dict(head_dim=272), -10), (dict(head_dim=0), -10), (dict(pages=0), -10), (dict(page_size=0), -10),
    (dict(table_pages=-1), -10), (dict(table_pages=1 << 27), -10), (dict(scale=float("nan")), -10),
    (dict(scale=float("inf")), -10), (dict(q_stride=(4, 8, 8)), -10), (dict(k_cache_stride=(-8, 8, 8)), -10),
    (dict(out_stride=(0, HQ * D, D)), -10), (dict(table_stride=-1), -10),
    (dict(q=None), -5), (dict(mask=None), -5), (dict(table=None), -5), (dict(workspace=None), -5),
    (dict(q=FAKE + 8), -6), (dict(k_cache=FAKE + 4 * 512 * MB + 2), -6), (dict(out=FAKE + 8 * 512 * MB + 4), -6),
    (dict(workspace_bytes=0), -11), (dict(out=FAKE + 64), -7), (dict(out=FAKE + 4 * 512 * MB), -7),
    (dict(workspace=FAKE + 512 * MB), -7), (dict(workspace=FAKE + 8 * 512 * MB), -7), (dict(batch=0, q=None), 0),
])
def test_library_refuses_attention(lib, bad, code):
    assert lib.tf_exl3_tree_attention(attention_args(lib, **bad), None) == code
    assert lib.tf_exl3_tree_attention(None, None) == -5


def test_attention_workspace_of_refused_sizes(lib):
    assert lib.tf_exl3_tree_attention_workspace(attention_args(lib)) > 0
    assert lib.tf_exl3_tree_attention_workspace(attention_args(lib, nodes=65)) == 0
    assert lib.tf_exl3_tree_attention_workspace(None) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(elem_bytes=8), -4), (dict(batch=-1), -10), (dict(tokens=-1), -10), (dict(kv_heads=0), -10),
    (dict(head_dim=0), -10), (dict(pages=0), -10), (dict(k_stride=(-1, 1, 1)), -10),
    (dict(v_cache_stride=(0, 64, 64)), -10), (dict(k=None), -5), (dict(table=None), -5), (dict(lengths=None), -5),
    (dict(k=FAKE + 1), -6), (dict(nodes=FAKE + 1), -6), (dict(k_cache=FAKE + 2), -7), (dict(batch=0, k=None), 0),
    (dict(tokens=0, k=None), 0), (dict(table_pages=0, k=None), 0),
])
def test_library_refuses_append(lib, bad, code):
    a = _lib.CacheAppendArgs(2, B, N, HKV, D, 5, PAGE, 2)
    for i, name in enumerate(("k", "v", "k_cache", "v_cache", "table", "lengths")):
        setattr(a, name, FAKE + i * MB)
    a.k_stride[:] = a.v_stride[:] = (N * HKV * D, HKV * D, D)
    a.k_cache_stride[:] = a.v_cache_stride[:] = (PAGE * HKV * D, HKV * D, D)
    a.table_stride = 2
    for name, value in bad.items():
        if name.endswith("_stride"):
            getattr(a, name)[:] = value
        else:
            setattr(a, name, value)
    assert lib.tf_exl3_cache_append(a, None) == code
    assert lib.tf_exl3_cache_append(None, None) == -5


def test_library_refuses_verification(lib):
    need = lib.tf_exl3_verify_workspace(B, N, V)
    assert need > 0 and lib.tf_exl3_verify_workspace(B, 1025, V) == 0 and lib.tf_exl3_verify_workspace(B, N, 0) == 0
    p = [FAKE + i * MB for i in range(12)]

    def tree(dtype=0, batch=B, nodes=N, vocab=V, logits=p[0], sb=N * V, sn=V, tokens=p[1], out=p[5], ws=p[8], n=need):
        return lib.tf_exl3_verify_tree(dtype, batch, nodes, vocab, logits, sb, sn, tokens, p[2], p[3], p[4], out, p[6],
                                       p[7], ws, n, None)

    def chain(dtype=0, batch=B, nodes=N, vocab=V, logits=p[0], sb=N * V, sn=V, tokens=p[1], out=p[5], ws=p[8], n=need):
        return lib.tf_exl3_verify_chain(dtype, batch, nodes, vocab, logits, sb, sn, tokens, p[2], N * V, V, p[3], p[4],
                                        out, p[6], ws, n, None)

    for call in (tree, chain):
        assert call(dtype=4) == -4
        assert call(batch=-1) == -10 and call(nodes=0) == -10 and call(nodes=1025) == -10 and call(vocab=0) == -10
        assert call(sb=-1) == -10 and call(sn=-8) == -10
        assert call(logits=None) == -5 and call(tokens=None) == -5 and call(ws=None) == -5 and call(out=None) == -5
        assert call(logits=p[0] + 2) == -6 and call(ws=p[8] + 8) == -6
        assert call(n=need - 1) == -11
        assert call(out=p[0] + 64) == -7 and call(out=p[6]) == -7 and call(ws=p[1]) == -7
        assert call(batch=0, logits=None) == 0


def test_library_refuses_distillation(lib):
    need = lib.tf_exl3_distill_workspace(0, 3, V, 5)
    assert need > 0 and lib.tf_exl3_distill_workspace(3, 3, V, 5) == 0 and lib.tf_exl3_distill_workspace(0, 3, V, 1025) == 0
    p = [FAKE + i * MB for i in range(8)]

    def call(dtype=0, rows=3, vocab=V, k=5, x=p[0], xs=V, index=p[1], top=p[2], tdt=0, w=p[3], t=1.0, loss=p[4],
             grad=p[5], gs=V, ws=p[6], n=need):
        return lib.tf_exl3_distill(dtype, rows, vocab, k, x, xs, index, top, tdt, w, t, loss, grad, gs, ws, n, None)

    assert call(dtype=5) == -4 and call(tdt=-1) == -4
    assert call(rows=-1) == -10 and call(vocab=0) == -10 and call(k=0) == -10 and call(k=1025) == -10
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        assert call(t=t) == -10
    assert call(xs=-1) == -10 and call(gs=V - 1) == -10
    assert call(x=None) == -5 and call(w=None) == -5 and call(loss=None, grad=None) == -5 and call(ws=None) == -5
    assert call(x=p[0] + 2) == -6 and call(grad=p[5] + 1) == -6 and call(ws=p[6] + 4) == -6
    assert call(n=need - 1) == -11
    assert call(grad=p[0] + 4) == -7 and call(loss=p[5]) == -7 and call(grad=p[2]) == -7
    assert call(rows=0, x=None) == 0


def test_argument_structures_have_the_headers_layout(lib):
    """The binding's structures against a C program's sizeof and offsetof."""
    import shutil
    import subprocess
    import tempfile
    from pathlib import Path

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    text = ['#include <stddef.h>', '#include <stdio.h>', '#include "tf_exl3.h"', 'int main(void) {']
    want = []
    for name, cls in (("tf_exl3_tree_attention_args", _lib.TreeAttentionArgs),
                      ("tf_exl3_cache_append_args", _lib.CacheAppendArgs)):
        text.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            text.append(f'printf("%zu\\n", offsetof({name}, {field}));')
            want.append(getattr(cls, field).offset)
    text.append("return 0; }")
    with tempfile.TemporaryDirectory() as d:
        src = Path(d) / "layout.c"
        src.write_text("\n".join(text))
        subprocess.run([cc, "-std=c11", f"-I{_lib.PKG.parent / 'include'}", str(src), "-o", f"{d}/layout"], check=True)
        got = subprocess.run([f"{d}/layout"], capture_output=True, text=True, check=True).stdout.split()
    assert [int(g) for g in got] == want
