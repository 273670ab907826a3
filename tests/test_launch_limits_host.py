"""Sizes whose launches would have 2^32 work-items or more are refused on the host before the first of a call's
launches. The pointers are never dereferenced, and no call here comes to a launch."""

import pytest
import torch  # noqa: F401

from tests.test_operators_host import FAKE, attention_args, lib  # noqa: F401
from trellis_quantized_linear_tf_amd import _lib

GB = 1 << 30
FAR = 1 << 44  # apart, whatever the extents


def at(i):
    return FAKE + i * FAR


@pytest.mark.parametrize("batch,nodes,vocab", [(16384, 1024, 1000), (65535, 1024, 5), (65535, 257, 2048)])
def test_trees_of_too_many_rows(lib, batch, nodes, vocab):  # noqa: F811
    need = max(lib.tf_exl3_verify_workspace(batch, nodes, vocab), 16)
    got = lib.tf_exl3_verify_tree(1, batch, nodes, vocab, at(0), nodes * vocab, vocab, at(1), at(2), at(3), None, at(4), at(5),
                                  at(6), at(7), need, None)
    assert got == -10


@pytest.mark.parametrize("batch,nodes,vocab", [(65535, 1024, 5000), (32, 512, 2 ** 31 - 1), (65535, 1024, 1025 * 2048)])
def test_too_many_chunks(lib, batch, nodes, vocab):  # noqa: F811
    assert lib.tf_exl3_verify_workspace(batch, nodes, vocab) == 0
    n = 1 << 62
    assert lib.tf_exl3_verify_tree(1, batch, nodes, vocab, at(0), 0, 0, at(1), at(2), at(3), None, at(4), at(5), at(6),
                                   at(7), n, None) == -10
    assert lib.tf_exl3_verify_chain(1, batch, nodes, vocab, at(0), 0, 0, at(1), at(2), 0, 0, at(3), None, at(4), at(5),
                                    at(6), n, None) == -10


def test_the_largest_number_of_chunks(lib):  # noqa: F811
    assert lib.tf_exl3_verify_workspace(65535, 1024, 2048) > 0
    assert lib.tf_exl3_verify_workspace(65535, 1024, 2049) == 0
    assert lib.tf_exl3_verify_workspace(4, 1, 2 ** 31 - 1) > 0


@pytest.mark.parametrize("dtype,rows,vocab", [(1, 1 << 24, 1000), (1, 1 << 23, 16400), (2, 1 << 22, 70000), (0, 1 << 24, 1),
                                              (0, (1 << 31) - 1, 3), (0, 1 << 23, 8200), (0, 1 << 22, 33000)])
def test_too_many_rows_of_distillation(lib, dtype, rows, vocab):  # noqa: F811
    need = max(lib.tf_exl3_distill_workspace(dtype, rows, vocab, 4), 16)
    got = lib.tf_exl3_distill(dtype, rows, vocab, 4, at(0), vocab, at(1), at(2), 0, at(3), 1.0, at(4), at(5), vocab, at(6),
                              need, None)
    assert got == -10


@pytest.mark.parametrize("batch,q_heads,kv_heads", [(65535, 512, 512), (65535, 65535, 65535), (2000, 65535, 3)])
def test_too_many_groups_of_attention(lib, batch, q_heads, kv_heads):  # noqa: F811
    kw = dict(batch=batch, nodes=64, q_heads=q_heads, kv_heads=kv_heads, pages=1, page_size=1, table_pages=1)
    a = attention_args(lib, **kw)
    a.workspace_bytes = 1 << 62
    for i, name in enumerate(("q", "k", "v", "mask", "k_cache", "v_cache", "table", "lengths", "out", "workspace")):
        setattr(a, name, at(i))
    a.out_stride[:] = 64 * q_heads * 64, q_heads * 64, 64
    assert lib.tf_exl3_tree_attention(a, None) == -10


def test_too_many_tokens_of_an_append(lib):  # noqa: F811
    a = _lib.CacheAppendArgs(1, 1, 1 << 30, 1, 5001, 1 << 20, 1 << 10, 1 << 20)
    for i, name in enumerate(("k", "v", "k_cache", "v_cache", "table", "lengths")):
        setattr(a, name, at(i))
    a.k_stride[:] = a.v_stride[:] = (0, 5001, 5001)
    a.k_cache_stride[:] = a.v_cache_stride[:] = (5001 << 10, 5001, 5001)
    a.table_stride = 1 << 20
    assert lib.tf_exl3_cache_append(a, None) == -10
