"""A dense-attention layer served over paged keys and values.

Three requests enter with their prompts and are decoded for some steps; every step
makes the same three calls:

    dsa_build_tables    pages for the new tokens, slots, positions, offsets
    dsa_rope_append     rotary positions; keys and values into the pages
    dsa_paged_attention the new tokens over everything cached

The projections around them are stand-ins (seeded random tensors).  At the end the
last step is checked against attention over the unpaged history.

    python examples/dense_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dsa_sparse_attention_step_gb300 as dsa  # noqa: E402

Q_HEADS, KV_HEADS, DIM, PAGES, MAX_PAGES = 16, 4, 128, 64, 16
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """The cache, its free pages and the requests' lengths between steps."""

    def __init__(self, requests):
        shape = (PAGES, KV_HEADS, 64, DIM)
        self.cache = dsa.KvCache(torch.zeros(shape, dtype=torch.bfloat16, device=DEV),
                                 torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
        freq = 10000.0 ** (-torch.arange(DIM // 2, dtype=torch.float64, device=DEV) / (DIM // 2))
        self.rope = dsa.Rope(freq)
        self.free = torch.randperm(PAGES, device=DEV).to(torch.int32)
        self.table = torch.zeros(requests, MAX_PAGES, dtype=torch.int32, device=DEV)
        self.lens = [0] * requests
        self.status = i32([0])

    def step(self, q, k, v, new):
        """Attention of the new tokens ([sum(new), heads, DIM] each) after they
        have been added to their requests."""
        tokens, n = sum(new), len(new)
        offsets, lens, taken = i32([0] * (n + 1)), i32([0] * n), i32([0])
        slots = torch.empty(tokens, dtype=torch.int64, device=DEV)
        positions = torch.empty(tokens, dtype=torch.int32, device=DEV)
        dsa.dsa_build_tables(i32(self.lens), i32(new), self.free, PAGES, self.table, offsets, lens,
                             slots, positions, None, taken, self.status)
        # the host knows the lengths, and so how many pages went
        before = sum(-(-a // 64) for a in self.lens)
        self.lens = [a + b for a, b in zip(self.lens, new)]
        self.free = self.free[sum(-(-a // 64) for a in self.lens) - before:].contiguous()

        turned = torch.empty_like(q)
        dsa.dsa_rope_append(self.cache, self.rope, positions, slots, q, k, v, turned, self.status)

        batch = dsa.Batch(offsets, lens, self.table, PAGES, self.lens, new)
        out = torch.empty_like(q)
        ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, self.cache, Q_HEADS),
                         dtype=torch.uint8, device=DEV)
        dsa.dsa_paged_attention(batch, self.cache, turned, DIM ** -0.5, out, None, ws, self.status)
        return out


def turn(x, freq):
    """Rotary positions 0 .. len(x) - 1 in float64."""
    angle = torch.arange(x.shape[0], device=DEV, dtype=torch.float64)[:, None] * freq
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x.double().chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)


def attend(q, k, v, freq):
    """The last token's attention over the whole history, in float64."""
    group = Q_HEADS // KV_HEADS
    q, k = turn(q, freq)[-1], turn(k, freq).repeat_interleave(group, dim=1)
    p = torch.softmax(torch.einsum("hd,shd->hs", q, k) * DIM ** -0.5, dim=-1)
    return torch.einsum("hs,shd->hd", p, v.double().repeat_interleave(group, dim=1))


def main(prompts=(70, 1, 300), steps=5):
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    server, history = Server(len(prompts)), [[] for _ in prompts]
    for new in [list(prompts)] + [[1] * len(prompts)] * steps:
        qkv = torch.randn(sum(new), Q_HEADS + 2 * KV_HEADS, DIM, generator=g, device=DEV)
        qkv = qkv.to(torch.bfloat16)
        out = server.step(*qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1), new)
        for past, part in zip(history, qkv.split(new)):
            past.append(part)
    assert int(server.status.item()) == 0
    worst = 0.0
    for b, past in enumerate(history):
        q, k, v = torch.cat(past).split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1)
        worst = max(worst, (out[b].double() - attend(q, k, v, server.rope.inv_freq)).abs().max().item())
    print("%d requests, %d tokens cached, %d pages left: largest difference %.2g" % (
        len(prompts), sum(server.lens), server.free.numel(), worst))
    return worst


if __name__ == "__main__":
    main()
