"""The operators between the projection's rows and the cache as a serving program runs them: prompts of
a packed batch through projection, norm and rotation, attention and the cache in 4 bits, then steps of drafted
trees over that cache. Every step is compared with the float64 oracle on the step's own inputs."""

import numpy as np
import pytest
import torch

import synth
import trellis_quantized_linear_tf_amd as tq
from oracle import operators as ops
from oracle import rows as oracle
from tests.test_gpu_norm_rotate import check as check_rotated
from tests.test_gpu_prompt_attention import check as check_prompt
from tests.test_gpu_tree_attention import tree_mask

pytestmark = pytest.mark.gpu

HQ, HKV, DIM, HIDDEN, PAGE = 4, 2, 64, 256, 16
HEADS = HQ + 2 * HKV
PARENTS = [-1, 0, 0, 1, 1]


def close(got, want, weight, spread, keys):
    h, f = 2.0 ** -8, 2.0 ** -24
    tol = h * np.abs(want) + (h + (2 * (DIM + 2) * spread[..., None] + keys + 64) * f) * weight + 2.0 ** -133
    over = np.abs(got.double().cpu().numpy() - want) - tol
    assert over.max() <= 0, over.max()


class Serving:
    def __init__(self, lengths, room=96):
        self.trellis = torch.from_numpy(synth.trellis_words(3, 4, HIDDEN, HEADS * DIM).view("int32").copy()).cuda()
        self.suh = torch.from_numpy(synth.signs(4, HIDDEN).view("float16").copy()).cuda()
        self.svh = torch.from_numpy(synth.signs(5, HEADS * DIM).view("float16").copy()).cuda()
        g = torch.Generator().manual_seed(1)
        self.weights = [(1 + 0.2 * torch.randn(DIM, generator=g)).bfloat16().cuda() for _ in range(2)]
        self.frequencies = (10000.0 ** (-torch.arange(0, DIM, 2) / DIM)).cuda()
        batch, cols = len(lengths), room // PAGE
        self.cache = [torch.full((batch * cols, HKV, PAGE, tq.q4_row_bytes(DIM)), 255, dtype=torch.uint8, device="cuda").transpose(1, 2)
                      for _ in range(2)]
        self.table = torch.randperm(batch * cols, generator=g).view(batch, cols).to(torch.int32).cuda()
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def rows(self, x, positions):
        """q, k, v of hidden rows, q and k normed and turned in place."""
        y = tq.project(x.flatten(0, -2), self.suh, self.trellis, self.svh, 4, HEADS * DIM, out_dtype=torch.bfloat16)
        y = y.view(*x.shape[:-1], HEADS, DIM)
        q, k, v = y.split([HQ, HKV, HKV], dim=-2)
        plain = y.cpu()
        tq.norm_rotate(q, k, positions, self.frequencies, *self.weights, out=(q, k))
        a, b, _ = plain.split([HQ, HKV, HKV], dim=-2)
        for got, was, w in ((q, a, self.weights[0]), (k, b, self.weights[1])):
            check_rotated(got, was, w.cpu(), positions.cpu(), self.frequencies.cpu(), 1e-6, False, "bf16")
        return q, k, v


@pytest.mark.parametrize("heads", ["strided", "own"])
def test_prompts_then_trees(gpu, heads):
    lengths = [37, 1, 20]
    s = Serving(lengths)
    g = torch.Generator().manual_seed(2)
    total, behind = sum(lengths), 6
    ends = [0, 37, 38, 58]
    x = torch.randn((total + behind, HIDDEN), generator=g).cuda()
    positions = torch.tensor([i for n in lengths for i in range(n)] + [0] * behind, dtype=torch.int32).cuda()
    q, k, v = s.rows(x, positions)
    if heads == "own":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    offsets = torch.tensor(ends, dtype=torch.int32).cuda()
    out = torch.zeros((total + behind, HQ, DIM), dtype=torch.bfloat16, device="cuda")
    tq.prompt_attention(q, k, v, offsets, out=out)
    check_prompt(out, torch.cat([q, k, v], 1).cpu(), [HQ, HKV, HKV], ends, "bf16")

    # The packed rows go into the cache as sequences of rows: row j of sequence b is token ends[b] + j.
    longest = max(lengths)
    at = torch.tensor([[min(b + j, total - 1) for j in range(longest)] for b in ends[:-1]]).cuda()
    counts = torch.tensor(lengths, dtype=torch.int32).cuda()
    tq.cache_append_q4(k[at], v[at], *s.cache, s.table, s.lengths, counts=counts)
    s.lengths += counts

    for step in range(3):
        hidden = torch.randn((3, len(PARENTS), HIDDEN), generator=g).cuda()
        depth = torch.tensor([bin(m).count("1") - 1 for m in tree_mask(PARENTS)], dtype=torch.int32).cuda()
        q, k, v = s.rows(hidden, s.lengths[:, None] + depth)
        mask = torch.tensor([tree_mask(PARENTS)] * 3).cuda()
        got = tq.tree_attention_q4(q, k, v, mask, *s.cache, s.table, s.lengths)
        values = tq.cache_read_q4(*s.cache, s.table, s.lengths, int(s.lengths.max()))
        n = values[0].shape[1]
        table = np.arange(3, dtype=np.int32)[:, None]  # one page a sequence
        f64 = [t.double().cpu().numpy() for t in (q, k, v, *values)]
        want, weight, spread = ops.tree_attention(*f64[:3], mask.cpu().numpy(), *f64[3:], table, s.lengths.cpu().numpy(), DIM ** -0.5)
        close(got, want, weight, spread, n + len(PARENTS))

        # The same attention over a cache in 16 bits that holds what was read.
        same = tq.tree_attention(q, k, v, mask, *values, torch.from_numpy(table).cuda(), s.lengths)
        close(same, want, weight, spread, n + len(PARENTS))

        accepted = torch.tensor([[0, 1, 3, -1, -1], [0, -1, -1, -1, -1], [0, 2, -1, -1, -1]], dtype=torch.int32).cuda()
        counts = torch.tensor([3, 1, 2], dtype=torch.int32).cuda()
        before = s.lengths.clone()
        tq.cache_append_q4(k, v, *s.cache, s.table, s.lengths, accepted, counts)
        s.lengths += counts
        back = tq.cache_read_q4(*s.cache, s.table, s.lengths, 3, first=before)
        for got, rows in zip(back, (k, v)):
            for b, path in enumerate(([0, 1, 3], [0], [0, 2])):
                stands = oracle.round_to(oracle.q4_unpack(oracle.q4_pack(rows[b, path].float().cpu().numpy())), "bf16")
                assert np.array_equal(got[b, : len(path)].double().cpu().numpy(), stands)
                assert not got[b, len(path):].any()


def test_on_another_stream(gpu):
    """The whole chain on a side stream, its results as on the default one."""
    results = []
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            s = Serving([30], room=64)
            x = torch.randn((30, HIDDEN), generator=torch.Generator().manual_seed(4)).cuda()
            q, k, v = s.rows(x, torch.arange(30, dtype=torch.int32, device="cuda"))
            out = tq.prompt_attention(q, k, v, torch.tensor([0, 30], dtype=torch.int32, device="cuda"))
            tq.cache_append_q4(k[None], v[None], *s.cache, s.table, s.lengths)
            s.lengths += 30
            tree = tq.tree_attention_q4(q[None, :2], k[None, :2], v[None, :2], torch.tensor([[1, 3]], device="cuda"), *s.cache,
                                        s.table, s.lengths)
            results.append((out.cpu(), tree.cpu(), tq.cache_read_q4(*s.cache, s.table, s.lengths, 30)[0].cpu()))
        torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b)
