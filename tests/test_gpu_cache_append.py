"""The paged cache's append on the GPU: every byte of both caches against the oracle."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import operators as ops
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def check(seed, batch, tokens, heads, dim, page, lengths, *, dtype=torch.int16, nodes=None, counts=None, heads_first=False,
          cols=None, edit=None, offset=0, stream=None):
    g = torch.Generator().manual_seed(seed)
    cols = -(-(max(lengths) + tokens) // page) if cols is None else cols
    pages = batch * cols + 2
    table = torch.randperm(pages, generator=g)[: batch * cols].view(batch, cols).to(torch.int32)
    if edit is not None:
        edit(table)
    raw = torch.randint(-100, 100, (batch, tokens, 2, heads, dim + offset), generator=g).to(torch.int16)
    kc, vc = (torch.randint(-100, 100, (pages, page, heads, dim), generator=g).to(torch.int16) for _ in range(2))
    narrow = torch.int8 if dtype.itemsize == 1 else torch.int16 if dtype.itemsize == 2 else torch.int32
    raw, kc, vc = (x.to(narrow) for x in (raw, kc, vc))
    rows = raw.cuda()[..., offset:]
    lengths = torch.tensor(lengths, dtype=torch.int32)
    want = ops.cache_append(raw[:, :, 0, :, offset:].numpy(), raw[:, :, 1, :, offset:].numpy(), kc.numpy(), vc.numpy(),
                            table.numpy(), lengths.numpy(), nodes, counts)

    def layout(c):
        c = c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if heads_first else c.cuda()
        return c.view(dtype)

    got = layout(kc), layout(vc)
    tq.cache_append(rows[:, :, 0].view(dtype), rows[:, :, 1].view(dtype), *got, table.cuda(), lengths.cuda(),
                    None if nodes is None else torch.from_numpy(nodes).cuda(),
                    None if counts is None else torch.from_numpy(counts).cuda())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert np.array_equal(a.view(narrow).cpu().numpy(), b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("dim", [1, 7, 64, 80, 128, 256])
def test_types_and_sizes(gpu, dtype, dim):
    say(f"append {dtype} {dim}")
    check(dim, 3, 5, 2, dim, 16, [0, 14, 33], dtype=dtype, heads_first=dim % 3 == 1)


@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 256])
@pytest.mark.parametrize("tokens", [1, 2, 17, 300])
def test_pages_and_tokens(gpu, page, tokens):
    say(f"append pages {page} {tokens}")
    check(page + tokens, 4, tokens, 3, 64, page, [0, page - 1, page, 2 * page + 1], heads_first=page == 16)


def test_rows_at_odd_addresses(gpu):
    check(1, 2, 9, 2, 64, 16, [3, 8], offset=1)
    check(2, 2, 9, 2, 63, 16, [3, 8], offset=4)


def test_accepted_nodes_and_counts(gpu):
    nodes = np.array([[0, 3, 5, -1, -1, -1], [0, -1, -1, -1, -1, -1], [0, 1, 2, 3, 4, 5]], np.int32)
    check(3, 3, 6, 4, 128, 16, [15, 0, 40], nodes=nodes, counts=np.array([3, 1, 6], np.int32))
    check(4, 3, 6, 4, 128, 16, [15, 0, 40], counts=np.array([0, 2, 6], np.int32))
    check(5, 3, 6, 4, 128, 16, [15, 0, 40], nodes=nodes[:, ::-1].copy())


def test_what_is_out_of_range_writes_nothing(gpu):
    nodes = np.array([[0, 6, -1, 2 ** 31 - 1, -(2 ** 31), 1]] * 3, np.int32)
    check(6, 3, 6, 2, 64, 16, [15, 0, 40], nodes=nodes, counts=np.array([99, -4, 6], np.int32))

    def edit(table):
        table[0, 0], table[1, 1], table[2, 0] = -1, 2 ** 31 - 1, table.numel() + 2
    check(7, 3, 40, 2, 64, 16, [0, 3, 9], edit=edit)
    check(8, 3, 40, 2, 64, 16, [0, 3, 9], cols=2)  # positions behind the table
    check(9, 3, 4, 2, 64, 16, [-3, 2 ** 31 - 1, 5], cols=2)


def test_offsets_past_32_bits(gpu):
    page, heads, dim = 16, 8, 128
    pages = (1 << 33) // (page * heads * dim * 2) * 9 // 8
    kc, vc = (torch.zeros((pages, page, heads, dim), dtype=torch.bfloat16, device=gpu) for _ in range(2))
    k, v = (torch.randn((1, 20, heads, dim), device=gpu, dtype=torch.bfloat16) for _ in range(2))
    table = torch.tensor([[pages - 1, pages // 2 + 1]], dtype=torch.int32, device=gpu)
    tq.cache_append(k, v, kc, vc, table, torch.tensor([3], dtype=torch.int32, device=gpu))
    torch.cuda.synchronize()
    for c, x in ((kc, k), (vc, v)):
        assert torch.equal(c[pages - 1, 3:], x[0, :13]) and torch.equal(c[pages // 2 + 1, :7], x[0, 13:])
        assert not c[pages - 1, :3].any() and not c[pages // 2 + 1, 7:].any() and not c[0].any()


def test_graph_replays_and_another_stream(gpu):
    kc, vc = (torch.zeros((8, 4, 2, 64), dtype=torch.bfloat16, device=gpu) for _ in range(2))
    k, v = (torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16, device=gpu) for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device=gpu).view(2, 4)
    lengths = torch.zeros(2, dtype=torch.int32, device=gpu)
    counts = torch.ones(2, dtype=torch.int32, device=gpu)
    args = (k, v, kc, vc, table, lengths, None, counts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.cache_append(*args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.cache_append(*args)
    for step in range(4):
        k.copy_(torch.randn(k.shape, device=gpu))
        v.copy_(torch.randn(v.shape, device=gpu))
        lengths.copy_(torch.tensor([step * 3, 5], device=gpu))
        counts.copy_(torch.tensor([3, step], device=gpu))
        torch.cuda.synchronize()
        before = [c.view(torch.int16).cpu().numpy() for c in (kc, vc)]
        graph.replay()
        torch.cuda.synchronize()
        want = ops.cache_append(k.view(torch.int16).cpu().numpy(), v.view(torch.int16).cpu().numpy(), *before,
                                table.cpu().numpy(), lengths.cpu().numpy(), None, counts.cpu().numpy())
        for c, w in zip((kc, vc), want):
            assert np.array_equal(c.view(torch.int16).cpu().numpy(), w)
