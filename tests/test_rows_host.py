"""Refusals of the operators between the projection's rows and the cache, on the host (no GPU): the
binding's chain of comparisons against its checks one by one, the GPU it makes current, the library's
own refusals with pointers that are never dereferenced. Nothing here launches a kernel."""

import ctypes
import random
import shutil
import subprocess

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.test_argument_checks_host import Near, change, refusal
from tests.test_operators_host import lib  # noqa: F401
from tests.test_other_gpu_host import Far, machine  # noqa: F401
from trellis_quantized_linear_tf_amd import _lib

bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8


def rotate():
    return dict(q=torch.zeros(2, 3, 4, 64, dtype=bf), k=torch.zeros(2, 3, 2, 64, dtype=bf), positions=torch.zeros(2, 3, dtype=i32),
                frequencies=torch.zeros(16), q_weight=torch.zeros(64, dtype=bf), k_weight=torch.zeros(64, dtype=bf))


def packed():
    a = rotate()
    return a | {n: a[n][0] for n in ("q", "k", "positions")}


def prompt():
    q, k = torch.zeros(6, 4, 64, dtype=bf), torch.zeros(6, 2, 64, dtype=bf)
    return dict(q=q, k=k, v=k.clone(), offsets=torch.zeros(3, dtype=i32), out=q.clone())


def append():
    k, cache = torch.zeros(2, 3, 2, 64, dtype=bf), torch.zeros(5, 16, 2, 40, dtype=u8)
    return dict(k=k, v=k.clone(), k_cache=cache, v_cache=cache.clone(), table=torch.zeros(2, 2, dtype=i32),
                lengths=torch.zeros(2, dtype=i32), nodes=torch.zeros(2, 3, dtype=i32), counts=torch.zeros(2, dtype=i32))


def read():
    a = append()
    return {n: a[n] for n in ("k_cache", "v_cache", "table", "lengths")} | dict(first=torch.zeros(2, dtype=i32))


def attention():
    a = append()
    q = torch.zeros(2, 3, 4, 64, dtype=bf)
    return dict(q=q, mask=torch.zeros(2, 3, dtype=torch.int64), out=q.clone()) | {
        n: a[n] for n in ("k", "v", "k_cache", "v_cache", "table", "lengths")}


def read_call(**kw):
    return tq.cache_read_q4(tokens=4, **kw)


CALLS = {"norm_rotate": (tq.norm_rotate, rotate), "norm_rotate packed": (tq.norm_rotate, packed),
         "prompt_attention": (tq.prompt_attention, prompt), "cache_append_q4": (tq.cache_append_q4, append),
         "cache_read_q4": (read_call, read), "tree_attention_q4": (tq.tree_attention_q4, attention)}


@pytest.mark.parametrize("name", CALLS)
def test_the_chain_accepts_what_the_checks_accept(machine, name):  # noqa: F811
    """As for the operators around the projection: a message that the checks give for tensors on the host is
    the one for tensors that say they are on a GPU, and where only their place was wrong there is none."""
    call, make = CALLS[name]
    r = random.Random(name)
    seen = {True: 0, False: 0}
    for _ in range(600):
        plain = make()
        for _ in range(r.choice([0, 1, 1, 1, 2])):
            n = r.choice([n for n, t in plain.items() if t is not None and t.dim() > 0])
            plain[n] = change(r, plain[n])
        said = {n: None if t is None else t.as_subclass(Near) for n, t in plain.items()}
        what = {n: None if t is None else (t.dtype, tuple(t.shape), t.stride()) for n, t in plain.items()}
        mine, its = refusal(call, said), refusal(call, plain)
        assert its is not None
        assert mine == (None if "must live on the GPU" in its else its), what
        seen[mine is None] += 1
    assert min(seen.values()) > 50


@pytest.mark.parametrize("name", CALLS)
def test_one_tensor_elsewhere(machine, name):  # noqa: F811
    call, make = CALLS[name]
    for n in make():
        for elsewhere, message in ((Far, "one GPU"), (torch.Tensor, "on the GPU")):
            args = {m: t.as_subclass(elsewhere if m == n else Near) for m, t in make().items()}
            assert message in (refusal(call, args) or ""), n


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_gpu_is_current_during_the_call(machine, name):  # noqa: F811
    call, make = CALLS[name]
    call(**{n: t.as_subclass(Far) for n, t in make().items()})
    assert [c[1:] for c in machine.calls] == [(1, 1001)] and machine.now == 0


@pytest.mark.parametrize("call,bad,message", [
    (tq.norm_rotate, dict(rotate(), eps=None), "weights belong to the norm"),
    (tq.norm_rotate, dict(rotate(), out=(torch.zeros(1),)), "out must be a pair"),
    (tq.norm_rotate, dict(rotate(), k_weight=torch.zeros(64)), "one element type"),
    (tq.norm_rotate, dict(rotate(), positions=torch.zeros(2, 3, dtype=torch.int64)), "positions must have element type"),
    (tq.norm_rotate, dict(rotate(), positions=None), "positions is required"),
    (tq.norm_rotate, dict(rotate(), q=torch.zeros(4, 64, dtype=bf)), "q must have 4 dimensions"),
    (tq.norm_rotate, dict(rotate(), out=(torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64, dtype=bf))), "q_out must have element"),
    (tq.prompt_attention, dict(prompt(), offsets=torch.zeros(0, dtype=i32)), "beginnings"),
    (tq.prompt_attention, dict(prompt(), k=torch.zeros(7, 2, 64, dtype=bf)), "k must have shape"),
    (tq.cache_append_q4, dict(append(), k_cache=torch.zeros(5, 16, 2, 64, dtype=bf)), "k_cache must have element type"),
    (tq.cache_append_q4, dict(append(), k_cache=torch.zeros(5, 16, 2, 64, dtype=u8)), "k_cache must have shape"),
    (tq.cache_append_q4, dict(append(), k=torch.zeros(2, 3, 2, 48, dtype=bf), v=torch.zeros(2, 3, 2, 48, dtype=bf)), "multiple of 32"),
    (read_call, dict(read(), k_cache=torch.zeros(5, 16, 2, 30, dtype=u8), v_cache=torch.zeros(5, 16, 2, 30, dtype=u8)), "q4_row_bytes"),
    (read_call, dict(read(), dtype=torch.float64), "dtype must be"),
    (tq.cache_read_q4, dict(read(), tokens=-1), "number of positions"),
    (tq.tree_attention_q4, dict(attention(), v_cache=torch.zeros(5, 16, 2, 60, dtype=u8)), "v_cache must have shape"),
])
def test_messages(call, bad, message):
    with pytest.raises(ValueError, match=message):
        call(**bad)


def test_row_bytes(lib):  # noqa: F811
    for dim in (32, 64, 96, 128, 256, 512, 4096):
        assert tq.q4_row_bytes(dim) == lib.tf_exl3_q4_row_bytes(dim) == dim * 5 // 8
    for dim in (0, 16, 48, -32, (1 << 24) + 32):
        assert lib.tf_exl3_q4_row_bytes(dim) == 0
        with pytest.raises(ValueError):
            tq.q4_row_bytes(dim)


# ---------------------------------------------------------------- the library's own refusals

FAKE, STEP = 0x7F0000000000, 1 << 28  # never dereferenced


def place(a, names, bad):
    for i, name in enumerate(names):
        setattr(a, name, FAKE + i * STEP)
    return bad


def fill(a, bad):
    for name, value in bad.items():
        if name.endswith("_stride") and isinstance(value, tuple):
            getattr(a, name)[:] = value
        else:
            setattr(a, name, value)
    return a


def rotate_args(**bad):
    a = _lib.NormRotateArgs(2, 2, 2, 3, 4, 2, 64, 32, 0, 1, 1e-6)
    place(a, ("q", "k", "q_weight", "k_weight", "positions", "frequencies", "q_out", "k_out"), bad)
    a.q_stride[:] = a.q_out_stride[:] = (768, 256, 64)
    a.k_stride[:] = a.k_out_stride[:] = (384, 128, 64)
    a.positions_stride = 3
    return fill(a, bad)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=3), -4), (dict(weight_dtype=-1), -4), (dict(batch=-1), -10), (dict(tokens=-1), -10),
    (dict(batch=1 << 12, tokens=1 << 12), -10), (dict(q_heads=0), -10), (dict(kv_heads=0), -10), (dict(q_heads=65536), -10),
    (dict(head_dim=8), -10), (dict(head_dim=72), -10), (dict(head_dim=528), -10), (dict(rotary_dim=8), -10),
    (dict(rotary_dim=80), -10), (dict(rotary_dim=-16), -10), (dict(eps=-1.0), -10), (dict(eps=float("nan")), -10),
    (dict(q_stride=(-1, 1, 1)), -10), (dict(k_stride=(1 << 32, 128, 64)), -10), (dict(q_out_stride=(0, 256, 64)), -10), (dict(positions_stride=-1), -10),
    (dict(q=None), -5), (dict(k_out=None), -5), (dict(positions=None), -5), (dict(frequencies=None), -5),
    (dict(q=FAKE + 1), -6), (dict(positions=FAKE + 4 * STEP + 2), -6), (dict(q_weight=FAKE + 2 * STEP + 1), -6),
    (dict(q_out=FAKE + 128), -7), (dict(q_out=FAKE, q_out_stride=(768, 256, 32)), -7), (dict(q_out=FAKE + STEP), -7),
    (dict(q_out=FAKE + 7 * STEP), -7), (dict(k_out=FAKE + 4 * STEP), -7), (dict(k_out=FAKE + 5 * STEP), -7),
    (dict(q_out=FAKE + 2 * STEP), -7), (dict(batch=0, q=None), 0), (dict(tokens=0, q=None), 0),
])
def test_library_refuses_norm_rotate(lib, bad, code):  # noqa: F811
    assert lib.tf_exl3_norm_rotate(rotate_args(**bad), None) == code
    assert lib.tf_exl3_norm_rotate(None, None) == -5


def test_rows_that_alternate_in_one_buffer(lib):  # noqa: F811
    """Refused only where heads meet: the call goes on to the launch, which has no GPU here."""
    row = 8 * 64
    strides = (3 * row, row, 64)
    kw = dict(q_stride=strides, k_stride=strides, q_out_stride=strides, k_out_stride=strides, q=FAKE, q_out=FAKE)
    assert lib.tf_exl3_norm_rotate(rotate_args(**kw, k=FAKE + 4 * 128 - 2, k_out=FAKE + 4 * 128 - 2), None) == -7
    assert lib.tf_exl3_norm_rotate(rotate_args(**kw, k=FAKE + 7 * 128, k_out=FAKE + 7 * 128), None) == -7  # into the next token
    short = kw | dict(q_stride=(2 * row, row, 64), q_out_stride=(2 * row, row, 64))
    assert lib.tf_exl3_norm_rotate(rotate_args(**short, k=FAKE + 4 * 128, k_out=FAKE + 4 * 128), None) == -7


def prompt_args(**bad):
    a = _lib.PromptAttentionArgs(2, 6, 2, 4, 2, 64, 0.125)
    place(a, ("q", "k", "v", "offsets", "out"), bad)
    a.q_stride[:] = a.out_stride[:] = (256, 64)
    a.k_stride[:] = a.v_stride[:] = (128, 64)
    return fill(a, bad)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=0), -4), (dict(dtype=3), -4), (dict(tokens=-1), -10), (dict(tokens=1 << 30), -10), (dict(batch=-1), -10),
    (dict(batch=1 << 30), -10), (dict(kv_heads=3), -10), (dict(kv_heads=0), -10), (dict(q_heads=65536, kv_heads=1), -10),
    (dict(head_dim=72), -10), (dict(head_dim=272), -10), (dict(scale=float("inf")), -10), (dict(q_stride=(4, 64)), -10),
    (dict(k_stride=((1 << 23) + 8, 64)), -10), (dict(v_stride=(-8, 64)), -10), (dict(out_stride=(0, 64)), -10),
    (dict(q_stride=(1 << 32, 64)), -10), (dict(tokens=(1 << 30) - 1, q_heads=65535, kv_heads=1), -10),
    (dict(q=None), -5), (dict(offsets=None), -5), (dict(k=FAKE + STEP + 8), -6), (dict(out=FAKE + 4 * STEP + 4), -6),
    (dict(out=FAKE), -7), (dict(out=FAKE + STEP + 64), -7), (dict(out=FAKE + 3 * STEP), -7), (dict(tokens=0, q=None), 0),
    (dict(batch=0, q=None), 0),
])
def test_library_refuses_prompt_attention(lib, bad, code):  # noqa: F811
    assert lib.tf_exl3_prompt_attention(prompt_args(**bad), None) == code
    assert lib.tf_exl3_prompt_attention(None, None) == -5


def cache_args(cls, names, **bad):
    a = cls(2, 2, 3, 2, 64, 5, 16, 2)
    place(a, names, bad)
    a.k_stride[:] = a.v_stride[:] = (384, 128, 64)
    a.k_cache_stride[:] = a.v_cache_stride[:] = (1280, 80, 40)
    a.table_stride = 2
    return fill(a, bad)


SHARED = [
    (dict(dtype=3), -4), (dict(batch=-1), -10), (dict(batch=65536), -10), (dict(tokens=-1), -10), (dict(tokens=(1 << 30) + 1), -10),
    (dict(kv_heads=0), -10), (dict(head_dim=48), -10), (dict(head_dim=0), -10), (dict(pages=0), -10), (dict(page_size=0), -10),
    (dict(table_pages=1 << 27), -10), (dict(k_cache_stride=(1280, 80, 42)), -10), (dict(k_stride=(-1, 1, 1)), -10),
    (dict(table_stride=-1), -10), (dict(k=None), -5), (dict(v_cache=None), -5), (dict(lengths=None), -5), (dict(table=None), -5),
    (dict(k=FAKE + 1), -6), (dict(k_cache=FAKE + 2), -6), (dict(tokens=0, k=None), 0), (dict(batch=0, k=None), 0),
]


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(k_cache=FAKE + 64), -7), (dict(v_cache=FAKE + 4 * STEP), -7), (dict(nodes=FAKE + 2 * STEP), -7),
    (dict(counts=FAKE + 3 * STEP), -7), (dict(k_cache_stride=(0, 80, 40)), -10), (dict(nodes=FAKE + 6 * STEP + 1), -6),
    (dict(table_pages=0, k=None), 0),
])
def test_library_refuses_append(lib, bad, code):  # noqa: F811
    a = cache_args(_lib.CacheAppendQ4Args, ("k", "v", "k_cache", "v_cache", "table", "lengths"), **bad)
    assert lib.tf_exl3_cache_append_q4(a, None) == code
    assert lib.tf_exl3_cache_append_q4(None, None) == -5


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(k_cache=FAKE + 4 * STEP), -7), (dict(k=FAKE + 2 * STEP), -7), (dict(v=FAKE + 4 * STEP + 128), -7),
    (dict(first=FAKE + 5 * STEP), -7), (dict(v_stride=(0, 128, 64)), -10), (dict(first=FAKE + 6 * STEP + 1), -6),
])
def test_library_refuses_read(lib, bad, code):  # noqa: F811
    a = cache_args(_lib.CacheReadQ4Args, ("k_cache", "v_cache", "table", "lengths", "k", "v"), **bad)
    assert lib.tf_exl3_cache_read_q4(a, None) == code
    assert lib.tf_exl3_cache_read_q4(None, None) == -5


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=80), -10), (dict(head_dim=48), -10), (dict(dtype=0), -4), (dict(nodes=65), -10), (dict(k_cache=FAKE + 4 * STEP + 2), -6),
    (dict(v_cache_stride=(1280, 80, 42)), -10), (dict(k_cache_stride=(1 << 32, 80, 40)), -10), (dict(out=FAKE + 4 * STEP), -7), (dict(workspace_bytes=0), -11), (dict(q=None), -5),
    (dict(batch=0, q=None), 0),
])
def test_library_refuses_attention(lib, bad, code):  # noqa: F811
    a = _lib.TreeAttentionArgs(2, 2, 3, 4, 2, 64, 5, 16, 2, 0.125)
    place(a, ("q", "k", "v", "mask", "k_cache", "v_cache", "table", "lengths", "out", "workspace"), bad)
    a.q_stride[:] = a.out_stride[:] = (768, 256, 64)
    a.k_stride[:] = a.v_stride[:] = (384, 128, 64)
    a.k_cache_stride[:] = a.v_cache_stride[:] = (1280, 80, 40)
    a.table_stride = 2
    a.workspace_bytes = lib.tf_exl3_tree_attention_q4_workspace(a)
    assert a.workspace_bytes > 0
    fill(a, bad)
    assert lib.tf_exl3_tree_attention_q4(a, None) == code
    assert lib.tf_exl3_tree_attention_q4(None, None) == -5
    assert (lib.tf_exl3_tree_attention_q4_workspace(a) > 0) == (code not in (-10, -4) or "v_cache_stride" in bad or "k_cache_stride" in bad)


def test_argument_structures_have_the_headers_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    text, want = ['#include <stddef.h>', '#include <stdio.h>', '#include "tf_exl3.h"', 'int main(void) {'], []
    for name, cls in (("norm_rotate", _lib.NormRotateArgs), ("prompt_attention", _lib.PromptAttentionArgs),
                      ("cache_append_q4", _lib.CacheAppendQ4Args), ("cache_read_q4", _lib.CacheReadQ4Args)):
        text.append(f'printf("%zu\\n", sizeof(tf_exl3_{name}_args));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            text.append(f'printf("%zu\\n", offsetof(tf_exl3_{name}_args, {field}));')
            want.append(getattr(cls, field).offset)
    src = tmp_path / "layout.c"
    src.write_text("\n".join([*text, "return 0; }"]))
    subprocess.run([cc, "-std=c11", f"-I{_lib.PKG.parent / 'include'}", str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(g) for g in got] == want


# Calls that are accepted go on to the launch: only where there is no GPU for it.
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch with addresses of nothing")

# Heads in front of tokens, [batch][heads][tokens][dim]: a sequence's queries, then its keys, in one buffer.
HEADS, TOKENS = (4, 2), 3
FIRST = dict(q_stride=(8 * TOKENS * 64, 64, TOKENS * 64), k_stride=(8 * TOKENS * 64, 64, TOKENS * 64))
FIRST |= dict(q_out_stride=FIRST["q_stride"], k_out_stride=FIRST["k_stride"], q=FAKE, q_out=FAKE)
BLOCK = HEADS[0] * TOKENS * 128  # bytes of a sequence's queries


@no_gpu
@pytest.mark.parametrize("behind,fine", [(0, True), (-2, False), (2 * TOKENS * 128, True), (2 * TOKENS * 128 + 2, False), (128, True)])
def test_heads_first_rows_that_alternate_in_one_buffer(lib, behind, fine):  # noqa: F811
    """Where they do not meet the call goes on to the launch, which has no GPU here."""
    k = FAKE + BLOCK + behind
    status = lib.tf_exl3_norm_rotate(rotate_args(**FIRST, k=k, k_out=k), None)
    assert status == (-9 if fine else -7)
    swapped = FIRST | dict(q=k, q_out=k, q_stride=FIRST["k_stride"], q_heads=HEADS[1], kv_heads=HEADS[0])
    assert lib.tf_exl3_norm_rotate(rotate_args(**swapped, k=FAKE, k_out=FAKE), None) == status


@no_gpu
def test_sequences_that_alternate_by_token(lib):  # noqa: F811
    """[tokens][heads][batch][dim]."""
    strides = (64, 8 * 2 * 64, 2 * 64)
    kw = dict(q_stride=strides, k_stride=strides, q_out_stride=strides, k_out_stride=strides, q=FAKE, q_out=FAKE)
    for k, status in ((4 * 256, -9), (4 * 256 - 2, -7), (6 * 256, -9), (6 * 256 + 2, -7)):
        assert lib.tf_exl3_norm_rotate(rotate_args(**kw, k=FAKE + k, k_out=FAKE + k), None) == status


@no_gpu
def test_alternating_rows_by_brute_force(lib):  # noqa: F811
    """Small buffers in every order of batch, tokens and heads with the keys at every place: refused wherever a byte is in a
    query row and in a key row, and accepted where each set fits behind the other within a step."""
    import itertools

    r = random.Random(5)
    accepted = 0
    for _ in range(400):
        batch, tokens, hq, hkv, dim = r.randint(1, 3), r.randint(1, 3), r.randint(1, 3), r.randint(1, 3), 16
        order = r.choice(list(itertools.permutations(range(3))))
        sizes = [batch, tokens, hq + hkv]
        strides, step = [0, 0, 0], dim
        for axis in reversed(order):
            strides[axis] = step
            step *= sizes[axis]
        at = r.choice([hq * strides[2], r.randrange(0, step)])

        def bytes_of(first, heads):
            return {first + b * strides[0] + t * strides[1] + h * strides[2] + d
                    for b in range(batch) for t in range(tokens) for h in range(heads) for d in range(dim)}

        meet = bool(bytes_of(0, hq) & bytes_of(at, hkv))
        kw = dict(q_stride=strides, k_stride=strides, q_out_stride=strides, k_out_stride=strides)
        kw = {n: tuple(s) for n, s in kw.items()}
        a = rotate_args(batch=batch, tokens=tokens, q_heads=hq, kv_heads=hkv, head_dim=dim, rotary_dim=16, q=FAKE, q_out=FAKE,
                        k=FAKE + 2 * at, k_out=FAKE + 2 * at, **kw)
        status = lib.tf_exl3_norm_rotate(a, None)
        assert status == -7 if meet else status in (-7, -9)
        if at == hq * strides[2]:
            assert not meet and status == -9, (order, sizes, hq)
        accepted += status == -9
    assert accepted > 100


@pytest.mark.parametrize("rotary", range(0, 66))
def test_rotary_sizes(lib, rotary):  # noqa: F811
    """Multiples of 8 from 16 on, or none."""
    fine = rotary == 0 or 16 <= rotary <= 64 and rotary % 8 == 0
    assert lib.tf_exl3_norm_rotate(rotate_args(rotary_dim=rotary, batch=0), None) == (0 if fine else -10)
