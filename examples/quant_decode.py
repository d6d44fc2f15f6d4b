"""A dense-attention layer served over an 8-bit cache whose scales follow the data.

As dense_decode.py, with INT8 (or E4M3) pages in place of 16-bit ones: half the memory, and
no scale to be known before the first token.  Every step makes three calls:

    dsa_build_tables    pages for the new tokens, slots, positions, offsets
    dsa_quant_append    rotary positions; keys and values quantised into the pages
    dsa_quant_attention the new tokens over everything cached

At the end dsa_quant_read gives back what the cache holds; the last step is checked against
attention over that, and what is held against what was written.

    python examples/quant_decode.py
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

    def __init__(self, requests, code):
        shape = (PAGES, KV_HEADS, 64, DIM)
        # nothing has to be initialised: a block's first token sets its scale
        self.cache = dsa.QuantCache(torch.empty(shape, dtype=code, device=DEV),
                                    torch.empty(shape, dtype=code, device=DEV),
                                    torch.empty(PAGES, KV_HEADS, 2, 4, device=DEV))
        freq = 10000.0 ** (-torch.arange(DIM // 2, dtype=torch.float64, device=DEV) / (DIM // 2))
        self.rope = dsa.Rope(freq)
        self.free = torch.randperm(PAGES, device=DEV).to(torch.int32)
        self.table = torch.zeros(requests, MAX_PAGES, dtype=torch.int32, device=DEV)
        self.lens = [0] * requests
        self.status = i32([0])

    def step(self, q, k, v, new):
        """Attention of the new tokens ([sum(new), heads, DIM] each) after they have been
        added to their requests, and their turned queries."""
        tokens, n = sum(new), len(new)
        offsets, lens, taken = i32([0] * (n + 1)), i32([0] * n), i32([0])
        slots = torch.empty(tokens, dtype=torch.int64, device=DEV)
        positions = torch.empty(tokens, dtype=torch.int32, device=DEV)
        dsa.dsa_build_tables(i32(self.lens), i32(new), self.free, PAGES, self.table, offsets, lens,
                             slots, positions, None, taken, self.status)
        before = sum(-(-a // 64) for a in self.lens)
        self.lens = [a + b for a, b in zip(self.lens, new)]
        self.free = self.free[sum(-(-a // 64) for a in self.lens) - before:].contiguous()

        turned = torch.empty_like(q)
        dsa.dsa_quant_append(self.cache, self.rope, positions, slots, q, k, v, turned, self.status)

        batch = dsa.Batch(offsets, lens, self.table, PAGES, self.lens, new)
        out = torch.empty_like(q)
        ws = torch.empty(dsa.dsa_quant_attention_workspace_size(batch, self.cache, Q_HEADS),
                         dtype=torch.uint8, device=DEV)
        dsa.dsa_quant_attention(batch, self.cache, turned, DIM ** -0.5, out, None, ws, self.status)
        return out, turned

    def held(self):
        """What the cache holds of every request: (keys, values) of all positions, in order."""
        offsets = [0]
        for n in self.lens:
            offsets.append(offsets[-1] + n)
        batch = dsa.Batch(i32(offsets), i32(self.lens), self.table, PAGES, self.lens, self.lens)
        k, v = torch.empty(2, offsets[-1], KV_HEADS, DIM, dtype=torch.float16, device=DEV)
        dsa.dsa_quant_read(batch, self.cache, k, v, self.status)
        return k.split(self.lens), v.split(self.lens)


def main(prompts=(70, 1, 300), steps=5, code=torch.int8):
    """(largest difference of the last step from attention over what is held, root mean
    square of what quantisation changed in the values, of unit size)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    server, history = Server(len(prompts), code), [[] for _ in prompts]
    for new in [list(prompts)] + [[1] * len(prompts)] * steps:
        qkv = torch.randn(sum(new), Q_HEADS + 2 * KV_HEADS, DIM, generator=g, device=DEV)
        qkv = qkv.to(torch.bfloat16)
        out, turned = server.step(*qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1), new)
        for past, part in zip(history, qkv.split(new)):
            past.append(part[:, -KV_HEADS:])
    keys, values = server.held()
    assert int(server.status.item()) == 0
    worst, group = 0.0, Q_HEADS // KV_HEADS
    for b, (k, v) in enumerate(zip(keys, values)):
        k, v = (x.double().repeat_interleave(group, dim=1) for x in (k, v))
        p = torch.softmax(torch.einsum("hd,shd->hs", turned[b].double(), k) * DIM ** -0.5, dim=-1)
        want = torch.einsum("hs,shd->hd", p, v)
        worst = max(worst, (out[b].double() - want).abs().max().item())
    lost = torch.cat([v.float() - torch.cat(past).float() for v, past in zip(values, history)])
    lost = lost.square().mean().sqrt().item()
    print("%d requests, %d tokens cached, %d pages left: largest difference %.2g, quantisation %.2g"
          % (len(prompts), sum(server.lens), server.free.numel(), worst, lost))
    return worst, lost


if __name__ == "__main__":
    main()
    main(code=torch.float8_e4m3fn)
