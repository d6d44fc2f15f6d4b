"""dsa_paged_attention where values, scores, batches and buffers are out of the ordinary."""
import copy

import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa
from test_gpu_paged_attention import BF16, DEV, FP8, Case

pytestmark = pytest.mark.gpu

def rows_of(c, b):
    return slice(c.offsets[b], c.offsets[b + 1])


def some_requests(c, order):
    """The case's requests `order` as a batch of their own over the same pages."""
    part = copy.copy(c)
    part.lens, part.new = [c.lens[b] for b in order], [c.new[b] for b in order]
    part.offsets = [0]
    for n in part.new:
        part.offsets.append(part.offsets[-1] + n)
    part.table = c.table[order].contiguous()
    part.q = torch.cat([c.q[rows_of(c, b)] for b in order])
    return part


@pytest.mark.parametrize("d,kv", [(64, BF16), (64, FP8), (128, BF16), (128, FP8), (256, BF16),
                                  (256, FP8)])
def test_batch_invariant_with_several_units_a_cta(d, kv):
    """300 requests of 2 to 9 pages and 8 KV heads, 2400 units: most begin after others in
    their CTA.  Bit for bit the same in another order, and alone."""
    lens = [65 + (b * 211) % 500 for b in range(300)]
    c = Case(lens, [1 + b % 3 for b in range(300)], 16, 8, d, BF16, kv, seed=40)
    prev = dsa.dsa_set_batch_invariant(True)
    try:
        out, lse = c.run()
        c.check(out, lse)
        order = [b * 77 % 300 for b in range(300)]
        other, other_lse = some_requests(c, order).run()
        want = torch.cat([torch.arange(c.offsets[b], c.offsets[b + 1]) for b in order]).to(DEV)
        assert torch.equal(other_lse, lse[want]) and torch.equal(other, out[want])
        for b in range(0, 300, 23):
            o, l = some_requests(c, [b]).run()
            assert torch.equal(l, lse[rows_of(c, b)]) and torch.equal(o, out[rows_of(c, b)])
    finally:
        dsa.dsa_set_batch_invariant(prev)
