"""Speculative decoding with trees of drafts, a one-layer model around the trellis
projection, on one GPU:

    python examples/speculative_decode.py [--steps 24] [--batch 4] [--temperature 0.0] [--cache-bits 4]

Each step drafts a tree with a small drafter, runs the tree's nodes through the model at
once (project, tree_attention), keeps the path that the model's own samples follow
(verify_tree), puts that path's keys and values into the paged cache (cache_append), and
teaches the drafter the model's top logits (distill). With temperature 0 the tokens are
those of decoding one by one, but where logits tie within the order of attention's fp32 sums,
which goes by the tree and the batch. With --cache-bits 4 (cache_append_q4, tree_attention_q4)
they may differ: a node sees the others of its tree as they are, and once they are accepted as
the cache holds them. Weights are random; the projections are 4-bit trellis streams.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
import trellis_quantized_linear_tf_amd as tq  # noqa: E402

DIM, Q_HEADS, KV_HEADS, HEAD_DIM, VOCAB, BITS = 512, 4, 2, 64, 1024, 4
PARENTS = [-1, 0, 0, 1, 1, 2, 2]  # two drafts a node, two levels deep
PAGE = 16
TOP = 16  # of the model's logits, for the drafter


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Projection:
    """A trellis projection in_dim -> out_dim with outputs of about the given size."""

    def __init__(self, seed, in_dim, out_dim, size, device):
        self.out_dim = out_dim
        words = synth.trellis_words(seed, BITS, in_dim, out_dim).view("int32")
        self.trellis = torch.from_numpy(words.copy()).to(device)
        self.suh = torch.from_numpy(synth.signs(seed + 1, in_dim).view("float16").copy()).to(device)
        signs = torch.from_numpy(synth.signs(seed + 2, out_dim).view("float16").copy()).to(device)
        one = torch.ones((1, in_dim), device=device)
        spread = tq.project(one, self.suh, self.trellis, signs, BITS, out_dim).square().mean().sqrt()
        self.svh = (signs.float() * size / spread).half()

    def __call__(self, x, dtype=torch.float32):
        return tq.project(x, self.suh, self.trellis, self.svh, BITS, self.out_dim, out_dtype=dtype)


class Model:
    def __init__(self, seed=1, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.device = torch.device(device)
        self.embedding = norm(torch.randn((VOCAB, DIM), generator=g)).to(device)
        heads = Q_HEADS + 2 * KV_HEADS
        self.qkv = Projection(seed * 100, DIM, heads * HEAD_DIM, 1.0, device)
        self.out = Projection(seed * 100 + 10, Q_HEADS * HEAD_DIM, DIM, 2.0, device)
        self.head = Projection(seed * 100 + 20, DIM, VOCAB, 4.0, device)

    def rows(self, tokens):
        """q, k, v [batch][nodes][heads][HEAD_DIM] of tokens [batch][nodes], and their embeddings."""
        x = self.embedding[tokens.long()]
        rows = self.qkv(x.flatten(0, 1), torch.bfloat16).view(*tokens.shape, -1, HEAD_DIM)
        return x, rows.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=2)

    def logits(self, x, attended):
        h = norm(x.flatten(0, 1) + self.out(attended.flatten(2).flatten(0, 1)))
        return self.head(h).view(*x.shape[:2], VOCAB)


class Cache:
    def __init__(self, batch, room, device, bits=16):
        per = -(-room // PAGE)
        self.bits = bits
        if bits == 4:  # a head's slots behind one another
            shape = (batch * per, KV_HEADS, PAGE, tq.q4_row_bytes(HEAD_DIM))
            self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=device).transpose(1, 2) for _ in range(2))
        else:
            shape = (batch * per, PAGE, KV_HEADS, HEAD_DIM)
            self.k, self.v = (torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2))
        g = torch.Generator().manual_seed(7)
        self.table = torch.randperm(batch * per, generator=g).view(batch, per).to(torch.int32).to(device)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=device)

    def append(self, k, v, nodes=None, counts=None):
        append = tq.cache_append_q4 if self.bits == 4 else tq.cache_append
        append(k, v, self.k, self.v, self.table, self.lengths, nodes, counts)
        self.lengths += k.shape[1] if counts is None else counts

    def attend(self, q, k, v, mask):
        attention = tq.tree_attention_q4 if self.bits == 4 else tq.tree_attention
        return attention(q, k, v, mask, self.k, self.v, self.table, self.lengths)


class Drafter:
    """Logits of the next token from the last one alone, trained while it drafts."""

    def __init__(self, device, rate=6.0):
        self.weight = torch.zeros((DIM, VOCAB), device=device)
        self.rate = rate

    def draft(self, model, last):
        """[batch][7] tokens of the tree under `last`."""
        tokens = [last]
        for node in (0, 1, 2):
            tokens += list((model.embedding[tokens[node].long()] @ self.weight).topk(2).indices.to(torch.int32).unbind(1))
        return torch.stack(tokens, 1)

    def learn(self, x, logits):
        """One step towards the model's top logits at every node; returns the mean loss before it."""
        x = x.flatten(0, 1)
        top = logits.flatten(0, 1).topk(TOP)
        weight = torch.full((x.shape[0],), 1.0 / x.shape[0], device=x.device)
        loss, grad = tq.distill(x @ self.weight, top.indices.to(torch.int32), top.values, weight)
        self.weight -= self.rate * x.shape[0] / DIM * (x.t() @ grad)
        return loss.mean()


def decode(model, prompt, tokens, trees=True, temperature=0.0, drafter=None, seed=3, cache_bits=16):
    """Continues prompt [batch][length] by at least `tokens` tokens a sequence. Returns the new tokens
    (a list a sequence), the steps taken and the drafter's losses."""
    batch = prompt.shape[0]
    parents = torch.tensor([PARENTS if trees else [-1]] * batch, dtype=torch.int32, device=model.device)
    nodes = parents.shape[1]
    seen = []
    for i, p in enumerate(PARENTS[:nodes]):
        seen.append(1 << i | (seen[p] if p >= 0 else 0))
    mask = torch.tensor([seen] * batch, dtype=torch.int64, device=model.device)
    heat = torch.full((batch,), temperature, device=model.device)
    g = torch.Generator(device=model.device).manual_seed(seed)
    cache = Cache(batch, prompt.shape[1] + (tokens + 1) * nodes, model.device, cache_bits)
    _, (_, k, v) = model.rows(prompt[:, :-1])
    cache.append(k, v)
    last = prompt[:, -1].to(torch.int32)
    drafter = drafter or Drafter(model.device)
    out, losses, steps = [[] for _ in range(batch)], [], 0
    while min(map(len, out)) < tokens:
        drafts = drafter.draft(model, last) if trees else last[:, None].contiguous()
        x, (q, k, v) = model.rows(drafts)
        logits = model.logits(x, cache.attend(q, k, v, mask))
        u = torch.rand((batch, nodes), generator=g, device=model.device)
        accepted, count, last = tq.verify_tree(logits, drafts, parents, u, heat)
        cache.append(k, v, accepted, count)
        if trees:
            losses.append(drafter.learn(x, logits))
        for b, (path, n, after) in enumerate(zip(accepted.tolist(), count.tolist(), last.tolist())):
            out[b] += [int(drafts[b, i]) for i in path[1:n]] + [after]
        steps += 1
    return out, steps, [float(x) for x in losses]


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=24, help="tokens a sequence, at least")
    parser.add_argument("--batch", type=int, default=4)
    parser.add_argument("--temperature", type=float, default=0.0)
    parser.add_argument("--cache-bits", type=int, choices=(16, 4), default=16)
    args = parser.parse_args()
    model = Model()
    g = torch.Generator().manual_seed(5)
    prompt = torch.randint(0, VOCAB, (args.batch, 21), generator=g).to(model.device)
    plain, plain_steps, _ = decode(model, prompt, args.steps, trees=False, temperature=args.temperature,
                                  cache_bits=args.cache_bits)
    drafter = Drafter(model.device)
    for run in range(3):
        got, steps, losses = decode(model, prompt, args.steps, temperature=args.temperature, drafter=drafter,
                                    cache_bits=args.cache_bits)
        same = [a[: args.steps] == b[: args.steps] for a, b in zip(got, plain)]
        print(f"run {run}: {steps} steps for {plain_steps} tokens, drafter's loss {losses[0]:.3f} -> {losses[-1]:.3f}, "
              f"as decoded one by one: {sum(same)} of {len(same)}")


if __name__ == "__main__":
    main()
