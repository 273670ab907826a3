"""The paged cache in 4 bits on the GPU: bytes written and values read are the oracle's, bit for bit."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import rows as oracle
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def setup(seed, dt, batch, tokens, heads, dim, page, lengths, *, heads_first=False, room=None, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rows = (torch.randn((batch, tokens, 2, heads, dim), generator=g) * spread).to(DT[dt])
    cols = room or -(-(max(lengths) + tokens) // page)
    pages = batch * cols + 2
    cache = torch.randint(0, 256, (2, pages, page, heads, dim // 8 * 5), generator=g, dtype=torch.uint8)
    table = torch.randperm(pages, generator=g)[: batch * cols].view(batch, cols).to(torch.int32)
    return rows[:, :, 0], rows[:, :, 1], cache, table, torch.tensor(lengths, dtype=torch.int32), heads_first


def on_gpu(cache, heads_first):
    return [c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if heads_first else c.cuda() for c in cache]


def append(k, v, cache, table, lengths, heads_first, nodes=None, counts=None):
    caches = on_gpu(cache, heads_first)
    kv = torch.stack([k, v], 2).cuda()  # rows of one projection
    up = [None if t is None else t.cuda() for t in (nodes, counts)]
    tq.cache_append_q4(kv[:, :, 0], kv[:, :, 1], *caches, table.cuda(), lengths.cuda(), *up)
    torch.cuda.synchronize()
    f = [t.float().numpy() for t in (k, v)]
    n = [None if t is None else t.numpy() for t in (nodes, counts)]
    want = oracle.cache_append_q4(*f, *cache.numpy(), table.numpy(), lengths.numpy(), *n)
    for got, w in zip(caches, want):
        assert np.array_equal(got.cpu().numpy(), w)
    return caches


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256, 512])
def test_append(gpu, dt, dim):
    say(f"append {dt} {dim}")
    append(*setup(dim, dt, 3, 5, 2, dim, 16, [0, 15, 33]))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages(gpu, page, heads_first):
    append(*setup(page, "bf16", 2, 70, 3, 64, page, [page, 2 * page - 1], heads_first=heads_first))


@pytest.mark.parametrize("batch,tokens,heads", [(1, 1, 1), (1, 2000, 1), (300, 1, 2), (2, 700, 5)])
def test_many_rows(gpu, batch, tokens, heads):
    append(*setup(tokens, "bf16", batch, tokens, heads, 64, 32, [i % 40 for i in range(batch)]))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("spread", [1e-8, 1e-6, 1e-4, 300.0, 1e4])
def test_sizes_of_numbers(gpu, dt, spread):
    """Down to scales that fp16 holds as subnormals or not at all, up to its largest numbers."""
    append(*setup(3, dt, 2, 40, 2, 64, 16, [3, 9], spread=spread))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_numbers_next_to_borders_and_none(gpu, dt):
    """Groups of few different numbers, whose quotients often lie between two codes; infinities and NaN."""
    k, v, cache, table, lengths, _ = setup(4, dt, 2, 64, 2, 64, 16, [3, 9])
    g = torch.Generator().manual_seed(9)
    k = (torch.randint(-30, 31, k.shape, generator=g) * 0.5).to(DT[dt])
    v = (torch.randint(0, 16, v.shape, generator=g) * 0.75 + torch.randint(0, 2, v.shape, generator=g) * 0.375).to(DT[dt])
    k[0, 3, 0, 5], k[0, 4, 1, 40], k[1, 5, 0, 0] = float("nan"), float("inf"), -float("inf")
    v[0, 0], v[0, 1] = 0.0, -0.0
    v[0, 2] = float("nan")
    append(k, v, cache, table, lengths, False)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_the_largest_numbers(gpu, dt):
    """fp16's largest numbers of both signs in a group: their bytes, and finite values in every type."""
    k, v, cache, table, lengths, _ = setup(14, dt, 1, 6, 1, 64, 16, [0])
    k[..., 0], k[..., 1], v[..., 40] = 65504.0, -65504.0, 65000.0
    k[0, 1] = k[0, 1].sign() * 65504.0
    caches = append(k, v, cache, table, lengths, False)
    for to in DT:
        for got in tq.cache_read_q4(*caches, table.cuda(), (lengths + 6).cuda(), 6, dtype=DT[to]):
            assert torch.isfinite(got).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_every_size_of_group(gpu, dt):
    """262144 groups of sizes and middles from 2^-40 to 2^17; one in eight has a number that is none or too large."""
    k, v, cache, table, lengths, _ = setup(15, dt, 2, 2048, 4, 128, 64, [5, 90])
    g = torch.Generator().manual_seed(16)
    for x in (k, v):
        groups = (*x.shape[:-1], x.shape[-1] // 32, 1)
        size, middle = (2.0 ** (torch.rand(groups, generator=g) * 57 - 40) for _ in range(2))
        middle *= torch.randint(-1, 2, groups, generator=g)
        y = torch.randn((*groups[:-1], 32), generator=g) * size + middle
        odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30, -1e30, 65450.0, -65500.0, 65408.0])
        at = torch.randint(0, 8 * 32, groups, generator=g)
        place = torch.arange(32) == at
        y = torch.where(place, odd[torch.randint(0, 8, groups, generator=g)], y)
        x.copy_(y.flatten(-2))
    append(k, v, cache, table, lengths, False)


def test_nodes_and_counts(gpu):
    k, v, cache, table, lengths, _ = setup(5, "bf16", 4, 6, 2, 64, 16, [0, 5, 17, 30])
    nodes = torch.tensor([[0, 2, 5, -1, -1, -1], [3, -1, 4, 9, 0, 1], [0, 1, 2, 3, 4, 5], [5, 5, 5, 5, 5, 5]], dtype=torch.int32)
    counts = torch.tensor([3, 6, -2, 99], dtype=torch.int32)
    append(k, v, cache, table, lengths, False, nodes, counts)


def test_what_lies_outside_is_not_written(gpu):
    k, v, cache, table, lengths, _ = setup(6, "bf16", 5, 8, 1, 64, 16, [28, 5, -3, 40, 2 ** 31 - 4], room=2)
    table[1] = torch.tensor([cache.shape[1], -1])
    append(k, v, cache, table, lengths, False)


def read(caches, cache, table, lengths, tokens, first, dt):
    up = None if first is None else first.cuda()
    got = tq.cache_read_q4(*caches, table.cuda(), lengths.cuda(), tokens, first=up, dtype=DT[dt])
    torch.cuda.synchronize()
    want = oracle.cache_read_q4(*cache.numpy(), table.numpy(), lengths.numpy(), tokens, None if first is None else first.numpy(), dt)
    for g, w in zip(got, want):
        assert g.dtype == DT[dt] and g.is_contiguous()
        assert np.array_equal(g.double().cpu().numpy(), w)


def filled(seed, heads, dim, page, lengths, heads_first=False, spread=1.0):
    """A cache with real rows in every slot."""
    _, _, cache, table, lengths, _ = setup(seed, "bf16", len(lengths), 1, heads, dim, page, lengths)
    r = np.random.default_rng(seed)
    for c in cache:
        x = r.standard_normal((*c.shape[:3], dim)).astype(np.float32) * spread
        c.copy_(torch.from_numpy(oracle.q4_pack(x)))
    return on_gpu(cache, heads_first), cache, table, lengths


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_read(gpu, dt, dim, heads_first):
    say(f"read {dt} {dim} {heads_first}")
    read(*filled(dim, 2, dim, 16, [0, 1, 40, 33], heads_first), 40, None, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("spread", [1e-7, 1e-5, 1e4])
def test_read_sizes_of_numbers(gpu, dt, spread):
    read(*filled(7, 2, 64, 16, [40], spread=spread), 40, None, dt)


def test_read_from_a_position(gpu):
    args = filled(8, 3, 64, 24, [50, 10, 70, 0, 33])
    read(*args, 30, torch.tensor([20, 0, -5, 3, 2 ** 31 - 10], dtype=torch.int32), "bf16")


def test_read_outside_gives_zeros(gpu):
    caches, cache, table, lengths = filled(9, 1, 64, 16, [33, 33, 33])
    table[1, 1], table[2, 0] = -4, cache.shape[1]
    lengths[0] = 5000
    read(caches, cache, table, lengths, 70, None, "f16")


@pytest.mark.parametrize("batch,tokens", [(1, 3000), (257, 3), (5, 600)])
def test_read_many(gpu, batch, tokens):
    read(*filled(batch, 2, 64, 32, [(tokens * (b + 1)) // batch for b in range(batch)]), tokens, None, "bf16")


def test_in_a_graph(gpu):
    """Append and read, captured once, replayed over other rows and lengths."""
    k, v, cache, table, lengths, _ = setup(11, "bf16", 3, 4, 2, 128, 16, [5, 0, 20])
    caches = on_gpu(cache, True)
    kg, vg, tg, lg = (t.contiguous().cuda() for t in (k, v, table, lengths))
    after = lg + 4
    stream = torch.cuda.Stream()

    def step():
        tq.cache_append_q4(kg, vg, *caches, tg, lg)
        return tq.cache_read_q4(*caches, tg, after, 4, first=lg)

    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = step()
    for seed in range(3):
        a = setup(20 + seed, "bf16", 3, 4, 2, 128, 16, [seed, 7 * seed, 20 - seed])
        kg.copy_(a[0]), vg.copy_(a[1]), lg.copy_(a[4])
        after.copy_(lg + 4)
        graph.replay()
        torch.cuda.synchronize()
        for got, x in zip(out, a[:2]):
            want = oracle.round_to(oracle.q4_unpack(oracle.q4_pack(x.float().numpy())), "bf16")
            assert np.array_equal(got.double().cpu().numpy(), want)


def test_nothing_to_do(gpu):
    k, v, cache, table, lengths, _ = setup(12, "bf16", 2, 3, 1, 64, 16, [0, 4])
    caches = on_gpu(cache, False)
    tq.cache_append_q4(k[:, :0].cuda(), v[:, :0].cuda(), *caches, table.cuda(), lengths.cuda())
    tq.cache_append_q4(k[:0].cuda(), v[:0].cuda(), *caches, table[:0].cuda(), lengths[:0].cuda())
    got = tq.cache_read_q4(*caches, table.cuda(), lengths.cuda(), 0)
    assert got[0].shape == (2, 0, 1, 64)
    for g, c in zip(caches, cache):
        assert torch.equal(g.cpu(), c)


def test_far_pages(gpu):
    """A head's row more than 2^32 bytes behind the cache's beginning."""
    page, heads, dim = 64, 1, 64
    pages = (1 << 32) // (page * heads * 40) + 10
    cache = torch.zeros((pages, page, heads, 40), dtype=torch.uint8, device="cuda")
    k = torch.randn((1, 5, 1, dim), generator=torch.Generator().manual_seed(1)).bfloat16()
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([3], dtype=torch.int32, device="cuda")
    other = torch.zeros((pages, page, heads, 40), dtype=torch.uint8, device="cuda")
    tq.cache_append_q4(k.cuda(), k.cuda(), cache, other, table, lengths)
    assert np.array_equal(cache[-1, 3:8].cpu().numpy(), oracle.q4_pack(k[0].float().numpy()))
    got = tq.cache_read_q4(cache, other, table, lengths + 5, 5, first=lengths)
    want = oracle.round_to(oracle.q4_unpack(oracle.q4_pack(k.float().numpy())), "bf16")
    assert np.array_equal(got[1].double().cpu().numpy(), want)
