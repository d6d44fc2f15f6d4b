"""dsa_quant_attention on the GPU against the definition in 64 bits.

Tolerances, per output value, from the arithmetic alone:
  - the output's rounding: half a step, eps / 2 of the value;
  - a probability times its block's scale rounded to f16: half a step, 2^-11 of sum p |v|;
    of those below 2^-29 of the row's largest, 2^-40 of that, times a code, per position
    (2^-26 and 2^-37 where the reference maximum may lag by a factor of eight);
  - a score's error e: fp32 dot products of D terms and the scale's product, (D + 9) 2^-23
    of the sum of the terms' sizes; it moves p by e, and out by 2 e sum p |v|;
  - a scale's logarithm: approximate to 2^-22 and added in fp32 to exponents below
    |z| log2 e + 48 + 15, so 2^-22 + 63 * 2^-24 < 2^-17 of sum p |v| beside what e covers,
    and as much in its sum;
  - fp32 sums over n positions and exponentials: n 2^-24 + 2^-20 of sum p |v|."""
import copy
import random

import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa
from paged_helpers import DEV, PAGE, attention_reference, ceil_pages
from quant_helpers import BLOCK, E4M3, INT8, decoded, random_cache, tables_of

pytestmark = pytest.mark.gpu

DEVICE_CHECK, TIMEOUT = 5, 6
BF16, F16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


class Case:
    """A batch over shuffled pages.  What no token may see is wild: pages that no request
    holds, rows past a context's end (NaN codes of E4M3, -128 of INT8) and the scales of
    blocks without a live row (NaN, infinite, 0).  far: a last request of one token, so long
    that the call is work enough for the tensor core kernel (9 * 10^9 operations; it takes
    requests of more than 32 rows, 48 of 64 dims, to a KV head)."""

    def __init__(self, lens, new, hq, hkv, d, dtype=BF16, code=E4M3, seed=0, q_scale=2.0,
                 far=False):
        lens, new = list(lens), list(new)
        if far:
            assert max(new) * (hq // hkv) > (48 if d == 64 else 32)
            lens.append(int(2.5e10 / (4.0 * (sum(new) + 1) * hq * d)) + 70)
            new.append(1)
        self.far = far
        g = torch.Generator(device=DEV)
        g.manual_seed(3000 + seed)
        self.lens, self.new, self.hq, self.d = list(lens), list(new), hq, d
        self.dtype, self.code = dtype, code
        self.table, self.pages = tables_of(g, lens, extra=3)
        self.k, self.v, self.scales = random_cache(g, self.pages, hkv, d, code)
        live = torch.zeros(self.pages, PAGE, dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            for i in range(ceil_pages(n)):
                live[int(self.table[b, i]), :min(PAGE, n - i * PAGE)] = True
        wild = 0x7f if code == E4M3 else 0x80
        for pool in (self.k, self.v):
            pool.view(torch.uint8).masked_fill_(~live[:, None, :, None], wild)
        dead = ~live.view(self.pages, -1, BLOCK).any(-1)[:, None, None, :].expand_as(self.scales)
        ends = torch.tensor([NAN, INF, 0.0, -1.0], device=DEV)
        self.scales = torch.where(dead, ends, self.scales)
        self.offsets = [0]
        for n in new:
            self.offsets.append(self.offsets[-1] + n)
        self.q = (q_scale * torch.randn(self.offsets[-1], hq, d, generator=g, device=DEV)).to(dtype)
        self.sm_scale = d ** -0.5

    def cache(self):
        return dsa.QuantCache(self.k, self.v, self.scales)

    def batch(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        return dsa.Batch(i32(self.offsets), i32(self.lens), self.table, self.pages, self.lens,
                         self.new)

    def run(self, q=None, status=0, batch=None):
        batch, cache = batch or self.batch(), self.cache()
        out = torch.full(self.q.shape, NAN, dtype=self.dtype, device=DEV)
        lse = torch.full(self.q.shape[:2], NAN, dtype=torch.float32, device=DEV)
        need = dsa.dsa_quant_attention_workspace_size(batch, cache, self.hq)
        if self.far:  # pieces of 128 rows
            assert need > 2 * 160 * 128 * self.d * 4
        ws = torch.full((need // 4 + (1 << 20),), NAN, dtype=torch.float32, device=DEV)
        ws[(need + 3) // 4:] = 7.0  # not part of it
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        dsa.dsa_quant_attention(batch, cache, self.q if q is None else q, self.sm_scale, out, lse,
                                ws, st)
        torch.cuda.synchronize()
        assert int(st.item()) == status
        assert (ws[(need + 3) // 4:] == 7.0).all()
        return out, lse

    def reference(self):
        k, v = (decoded(x, self.scales, i) for i, x in enumerate((self.k, self.v)))
        return attention_reference(self.q, k, v, 1.0, 1.0, self.sm_scale, self.offsets, self.lens,
                                   self.table, self.pages)

    def tolerances(self, r):
        n = max(self.lens + [1])
        e = (self.d + 9) * 2.0**-23 * r["terms"]
        fine = torch.isfinite(self.scales)
        largest = float(torch.where(fine, self.scales, 0.0).max()) * 448
        tol = (torch.finfo(self.dtype).eps / 2 * r["out"].abs() +
               (2.0**-11 + 2.0**-16 + n * 2.0**-24 + 2.0**-20 + 2 * e)[..., None] * r["mean_abs"] +
               n * 2.0**-37 * largest)
        if self.dtype == F16:
            tol += 2.0**-25
        lse = torch.where(torch.isinf(r["lse"]), 0.0, r["lse"])
        return tol, e + 2.0**-16 + n * 2.0**-24 + 2.0**-20 + 2.0**-22 * lse.abs()

    def check(self, out, lse):
        r = self.reference()
        tol, lse_tol = self.tolerances(r)
        err = (out.double() - r["out"]).abs()
        assert (err <= tol).all(), float((err / tol.clamp_min(1e-30)).max())
        empty = torch.isinf(r["lse"])
        assert torch.equal(torch.isneginf(lse), empty)
        off = (torch.where(empty, 0.0, lse.double()) - torch.where(empty, 0.0, r["lse"])).abs()
        assert (off <= lse_tol).all()

    def part(self, order):
        """The requests `order` as a batch of their own over the same pages."""
        c = copy.copy(self)
        c.far = False
        c.lens, c.new = [self.lens[b] for b in order], [self.new[b] for b in order]
        c.offsets = [0]
        for n in c.new:
            c.offsets.append(c.offsets[-1] + n)
        c.table = self.table[order].contiguous()
        c.q = torch.cat([self.q[self.offsets[b]:self.offsets[b + 1]] for b in order])
        return c


def spread(seed, requests, top):
    rng = random.Random(seed)
    return [rng.randint(1, top) for _ in range(requests - 1)] + [top]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,new", [(1, 1, 1), (12, 1, 1), (32, 8, 5), (40, 2, 1), (8, 1, 9),
                                        (15, 3, 27)])
@pytest.mark.parametrize("filler,top", [(0, 1500), (170, 2100), (170, 300)])
def test_formats_and_head_layouts(dtype, code, d, hq, hkv, new, filler, top):
    """Few requests, and more than there are SMs, most of one token: every plan."""
    lens = [max(n, new) for n in spread(d + hq, 5, top)] + [1] * filler
    c = Case(lens, [new] * 5 + [1] * filler, hq, hkv, d, dtype, code, seed=hq)
    c.check(*c.run())


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 33, 47, 48, 63, 64, 65, 127, 129, 257])
@pytest.mark.parametrize("new,code", [(1, E4M3), (1, INT8), (7, E4M3), (7, INT8)])
def test_lengths(length, new, code):
    c = Case([length, 3 * length], [min(new, length), 1], 4, 2, 128, BF16, code, seed=length)
    c.check(*c.run())
    for d in (64, 256):
        c = Case([length, 3 * length] * 45, [min(new, length), 1] * 45, 4, 2, d, BF16, code,
                 seed=length)
        c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,d,length,new,code", [
    (4, 1, 128, 70001, 1, E4M3), (3, 3, 64, 33333, 3, INT8), (12, 1, 256, 20011, 4, INT8),
    (8, 1, 256, 60011, 5, E4M3), (24, 1, 128, 60019, 1, INT8), (48, 1, 128, 60021, 1, E4M3),
    (64, 1, 64, 60023, 1, INT8)])
def test_one_long_request_is_split_and_joined(hq, hkv, d, length, new, code):
    c = Case([length], [new], hq, hkv, d, BF16, code, seed=length)
    c.check(*c.run())


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("lens,new,hq,hkv,d", [
    ([333, 200, 90], [333, 60, 1], 6, 2, 128), ([1500], [700], 8, 2, 128),
    ([130, 65], [130, 1], 4, 4, 64), ([700, 1000], [129, 255], 3, 1, 256),
    ([2048, 64, 5], [1, 64, 5], 16, 4, 128), ([1025], [1025], 16, 1, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("far", [False, True])
def test_prompts(lens, new, hq, hkv, d, dtype, code, far):
    c = Case(lens, new, hq, hkv, d, dtype, code, seed=8, far=far)
    c.check(*c.run())


@pytest.mark.parametrize("dtype,code", [(BF16, E4M3), (F16, E4M3), (BF16, INT8), (F16, INT8)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,new", [(32, 8, 13), (40, 2, 3), (8, 1, 9), (3, 3, 60), (64, 1, 2)])
@pytest.mark.parametrize("filler,top", [(0, 1500), (170, 300)])
def test_tensor_core_formats_and_head_layouts(dtype, code, d, hq, hkv, new, filler, top):
    """Several requests of many rows among requests of one token, of every length of a step."""
    lens = [max(n, new) for n in spread(d + hq, 7, top)] + [1 + 13 * b for b in range(filler)]
    c = Case(lens, [new] * 7 + [1] * filler, hq, hkv, d, dtype, code, seed=hq, far=True)
    c.check(*c.run())


@pytest.mark.parametrize("length", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 193, 257, 385])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tensor_core_lengths(length, d):
    for code in (E4M3, INT8):
        c = Case([length, 3 * length, 700], [min(30, length), 1, 50], 8, 2, d, BF16, code,
                 seed=length, far=True)
        c.check(*c.run())


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("copies", [1, 60])
def test_rows_that_see_nothing(code, copies):
    """Padding requests, tokens before position 0, requests without new tokens."""
    lens, new = [0, 100, 0, 3, 2, 500], [1, 2, 5, 6, 3, 0]
    c = Case(lens * copies, new * copies, 8, 2, 128, BF16, code, seed=2)
    out, lse = c.run()
    c.check(out, lse)
    for rows in (slice(0, 1), slice(3, 8), slice(8, 11), slice(14, 15)):
        assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()


@pytest.mark.parametrize("d,code", [(64, INT8), (128, E4M3), (128, INT8), (256, E4M3)])
@pytest.mark.parametrize("copies", [1, 40])
def test_tensor_core_rows_that_see_nothing(d, code, copies):
    lens, new = [0, 100, 0, 3, 2, 500, 130], [1, 20, 50, 60, 3, 0, 300]
    c = Case(lens * copies, new * copies, 8, 2, d, BF16, code, seed=2, far=True)
    out, lse = c.run()
    c.check(out, lse)
    for rows in (slice(0, 1), slice(21, 71), slice(71, 128), slice(131, 132), slice(134, 304)):
        assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("d,lens,hq,hkv,far", [
    (128, [700, 90], 8, 2, False), (64, [300] * 200, 4, 1, False), (128, [2500] * 170, 4, 1, False),
    (256, [1500] * 10, 24, 1, False), (64, [900, 5000], 64, 1, True), (128, [900, 5000], 40, 1, True),
    (256, [900, 5000], 40, 1, True)])
def test_scales_far_apart(code, d, lens, hq, hkv, far):
    """Blocks whose values' scales spread over 2^-40 .. 2^6 and a sink, a first position
    that draws most of the probability and whose value is nearly 0: what the others give
    keeps its accuracy."""
    c = Case(lens, [1] * len(lens), hq, hkv, d, BF16, code, seed=31, far=far)
    lens = c.lens
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    spread_ = torch.randint(-40, 7, c.scales[:, :, 1].shape, generator=g, device=DEV)
    fine = torch.isfinite(c.scales[:, :, 1]) & (c.scales[:, :, 1] > 0)
    c.scales[:, :, 1] = torch.where(fine, torch.exp2(spread_.float()), c.scales[:, :, 1])
    first = c.table[:, 0].long()
    c.scales[first, :, 1, 0] = 2.0**-45
    c.q[:, :, 0] = 40.0
    c.k.view(torch.uint8)[first, :, 0, 0] = 0x7e if code == E4M3 else 127
    out, lse = c.run()
    r = c.reference()
    e = (d + 9) * 2.0**-23 * r["terms"]
    n = max(lens)
    # relative to sum p |v| alone: whatever the largest scale of all
    tol = (torch.finfo(BF16).eps / 2 * r["out"].abs() +
           (2.0**-11 + 2.0**-16 + n * 2.0**-24 + 2.0**-20 + 2 * e)[..., None] * r["mean_abs"])
    # products below 2^-26 of the row's largest one, which is at most sum p |v| / |code| times
    # the codes: 2^-37 n of the row's largest mean_abs, times the largest code over 1
    tol += n * 2.0**-37 * 448 * r["mean_abs"].amax(-1, keepdim=True)
    err = (out.double() - r["out"]).abs()
    assert (err <= tol).all(), float((err / tol).max())
    off = (lse.double() - r["lse"]).abs()
    assert (off <= e + 2.0**-16 + n * 2.0**-24 + 2.0**-22 * r["lse"].abs()).all()


@pytest.mark.parametrize("code", [E4M3, INT8])
def test_scales_outside_their_range_count_as_its_ends(code):
    c = Case([130, 64], [1, 2], 4, 2, 64, BF16, code, seed=32)
    page = c.table[:, 0].long()
    want = copy.copy(c)
    want.scales = c.scales.clone()
    for block, bad, end in ((0, NAN, 2.0**-48), (1, -1.0, 2.0**-48), (2, 0.0, 2.0**-48)):
        c.scales[page, :, :, block] = bad
        want.scales[page, :, :, block] = end
    out, lse = c.run()
    want.check(out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,new", [([200, 130, 67], [5, 3, 4]), ([200, 130, 67] * 60, [5, 3, 4] * 60),
                                      ([2900, 1300, 64, 700] * 12, [5, 2, 4, 1] * 12),
                                      ([150, 400], [150, 300])])
@pytest.mark.parametrize("far", [False, True])
def test_nan_codes_reach_the_rows_that_see_them(lens, new, d, far):
    """E4M3: the last new token's value is NaN in one dim of each head.  Earlier tokens'
    rows are as if it were not there."""
    hq, hkv = 8, 2
    if far and max(new) < 20:
        lens, new = lens + [300], new + [20]
    c = Case(lens, new, hq, hkv, d, BF16, E4M3, seed=43, far=far)
    lens, new = c.lens, c.new
    r = c.reference()
    tol, lse_tol = c.tolerances(r)
    want = r["out"].clone()
    for b, length in enumerate(lens):
        at = length - 1
        for h in range(hkv):
            dim = (5 * b + h) % d
            c.v.view(torch.uint8)[int(c.table[b, at // PAGE]), h, at % PAGE, dim] = 0x7f
            if new[b] > 1:
                want[c.offsets[b + 1] - 1, 4 * h:4 * h + 4, dim] = NAN
            else:
                want[c.offsets[b], 4 * h:4 * h + 4, dim] = NAN
    out, lse = c.run()
    assert torch.equal(out.isnan(), want.isnan())
    err = torch.where(want.isnan(), 0.0, out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp_min(1e-30)).max())
    assert ((lse.double() - r["lse"]).abs() <= lse_tol).all()


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("far", [False, True])
def test_a_row_of_nan_stays_alone(code, far):
    c = Case([300, 90, 400], [3, 1, 200], 8, 2, 128, BF16, code, seed=21, far=far)
    want, want_lse = c.run()
    c.q[1, 2, 5] = NAN
    out, lse = c.run()
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
    out[1, 2], lse[1, 2] = want[1, 2], want_lse[1, 2]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("d,more", [(64, 0), (64, 40), (128, 40), (256, 40)])
def test_queries_of_extreme_size(code, d, more):
    c = Case([600, 601, 602] + [500] * (more > 0), [1, 1, 1] + [more] * (more > 0), 4, 2, d, BF16,
             code, seed=7, far=more > 0)
    c.q[0] *= 2.0**20
    c.q[1] *= 2.0**-30
    c.q[2, :, ::2] *= 2.0**-20
    c.sm_scale = 2.0**-22
    c.check(*c.run())
    c.q *= 2.0**-60  # all scores 0; positions past a row's view stay masked
    c.sm_scale = 2.0**-100
    c.check(*c.run())


@pytest.mark.parametrize("new,far", [([1, 2], False), ([1, 200], False), ([1, 200], True)])
def test_pages_outside_the_pool_are_left_out_and_reported(new, far):
    c = Case([700, 300], new, 8, 2, 128, BF16, INT8, seed=9, far=far)
    for b, i, page in ((0, 0, -1), (0, 7, c.pages), (1, 4, 1 << 30)):
        c.table[b, i] = page
    out, lse = c.run(status=DEVICE_CHECK)
    c.check(out, lse)


@pytest.mark.parametrize("new,far", [(1, False), (70, False), (70, True)])
def test_requests_that_contradict_the_host_sizes_are_reported_and_not_written(new, far):
    c = Case([200, 300, 164], [new] * 3, 4, 2, 64, BF16, E4M3, seed=10, far=far)
    b = c.batch()
    b.seq_lens[1] = 1 << 24
    out, lse = c.run(status=DEVICE_CHECK, batch=b)
    rows = slice(new, 2 * new)
    assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    # the others as ever (to the last bit only where the plan runs them whole: without the
    # second request the list is cut in other places)
    r = c.reference()
    tol, lse_tol = c.tolerances(r)
    keep = [t for t in range(3 * new) if not new <= t < 2 * new]
    assert ((out.double() - r["out"]).abs() <= tol)[keep].all()
    assert ((lse.double() - r["lse"]).abs() <= lse_tol)[keep].all()


@pytest.mark.parametrize("lens,new,far", [([130, 700], [2, 1], False), ([130, 700], [2, 300], False),
                                          ([130, 700], [2, 300], True)])
def test_queries_as_a_slice_of_a_projection(lens, new, far):
    c = Case(lens, new, 8, 2, 128, BF16, INT8, seed=11, far=far)
    wide = torch.full((c.offsets[-1], 12, 128), NAN, dtype=BF16, device=DEV)
    wide[:, 2:10] = c.q
    out, _ = c.run(q=wide[:, 2:10])
    same, _ = c.run()
    assert torch.equal(out, same)


@pytest.mark.parametrize("lens,new,hq,hkv,d,code", [
    ([150000, 99000], [1, 1], 32, 8, 128, INT8), ([150000, 99000], [6, 6], 16, 4, 128, E4M3),
    ([50000, 9000], [1, 1], 8, 4, 256, INT8), ([3000, 5000], [600, 1000], 8, 2, 128, E4M3),
    ([3000, 5000], [600, 1000], 8, 2, 64, INT8), ([3000, 5000], [600, 1000], 8, 2, 256, INT8)])
def test_calls_in_a_row_give_the_same_results(lens, new, hq, hkv, d, code):
    """Passes that follow one another without a wait, the workspace shared."""
    c = Case(lens, new, hq, hkv, d, BF16, code, seed=18)
    want, want_lse = c.run()
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_quant_attention_workspace_size(batch, cache, hq), dtype=torch.uint8,
                     device=DEV)
    outs = [(torch.zeros_like(want), torch.zeros_like(want_lse)) for _ in range(8)]
    for out, lse in outs:
        dsa.dsa_quant_attention(batch, cache, c.q, c.sm_scale, out, lse, ws)
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    c.check(want, want_lse)


@pytest.mark.parametrize("d,code", [(64, E4M3), (128, INT8), (256, E4M3)])
def test_batch_invariant_switch(d, code):
    """Under the switch a request's results do not depend on its batch, bit for bit."""
    lens = [65 + (b * 211) % 500 for b in range(120)] + [3000]
    new = [1 + b % 3 for b in range(120)] + [300]
    c = Case(lens, new, 16, 4, d, BF16, code, seed=40)
    prev = dsa.dsa_set_batch_invariant(True)
    try:
        out, lse = c.run()
        c.check(out, lse)
        order = [b * 50 % 121 for b in range(121)]
        other, other_lse = c.part(order).run()
        want = torch.cat([torch.arange(c.offsets[b], c.offsets[b + 1]) for b in order]).to(DEV)
        assert torch.equal(other_lse, lse[want]) and torch.equal(other, out[want])
        for b in (0, 23, 70, 120):
            o, l = c.part([b]).run()
            rows = slice(c.offsets[b], c.offsets[b + 1])
            assert torch.equal(l, lse[rows]) and torch.equal(o, out[rows])
    finally:
        dsa.dsa_set_batch_invariant(prev)


@pytest.mark.parametrize("new,far", [([1, 3], False), ([1, 400], False), ([1, 400], True)])
def test_on_another_stream_and_in_a_graph(new, far):
    c = Case([3000, 650], new, 8, 2, 128, BF16, INT8, seed=14, far=far)
    want, want_lse = c.run()
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_quant_attention_workspace_size(batch, cache, 8), dtype=torch.uint8,
                     device=DEV)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsa.dsa_quant_attention(batch, cache, c.q, c.sm_scale, out, lse, ws, None, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_quant_attention(batch, cache, c.q, c.sm_scale, out, None, ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("new,far", [(2, False), (300, False), (300, True)])
def test_pool_offsets_beyond_32_bits(new, far):
    """Pools of more than 2^32 bytes, their last pages in use."""
    c = Case([1000], [new], 8, 8, 128, BF16, INT8, seed=15, far=far)
    want, want_lse = c.run()
    n = c.pages
    pages = (1 << 32) // (8 * PAGE * 128) + 40
    pool = torch.empty(pages, 8, PAGE, 128, dtype=INT8, device=DEV)
    scales = torch.empty(pages, 8, 2, 4, dtype=torch.float32, device=DEV)
    pool[pages - n:], scales[pages - n:] = c.k, c.scales
    low = copy.copy(c)
    low.v = low.k
    want, want_lse = low.run()
    c.table = c.table + (pages - n)
    c.k = c.v = pool
    c.scales, c.pages = scales, pages
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("lens,new,far", [([900, 300], [1, 1], False), ([300, 2000], [30, 60], True)])
def test_a_wait_that_runs_out_is_reported_and_the_stream_recovers(lens, new, far):
    c = Case(lens, new, 8, 2, 128, BF16, INT8, seed=22, far=far)
    want, want_lse = c.run()
    batch, cache, out = c.batch(), c.cache(), torch.empty_like(want)
    ws = torch.empty(dsa.dsa_quant_attention_workspace_size(batch, cache, c.hq),
                     dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsa.dsa_test_quant_attention_wait_timeout(batch, cache, c.q, c.sm_scale, out, None, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == TIMEOUT
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_python_checks():
    c = Case([300, 64], [1, 1], 4, 2, 64, BF16, INT8, seed=17)
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_quant_attention_workspace_size(batch, cache, 4), dtype=torch.uint8,
                     device=DEV)
    out = torch.empty_like(c.q)
    for bad in (dict(q=c.q[:1]), dict(q=c.q.float()), dict(q=c.q[..., ::2]), dict(out=out[:1]),
                dict(out=out.half()), dict(lse=torch.empty(3, device=DEV)),
                dict(out=torch.empty(4, 2, 64, dtype=BF16, device=DEV))):
        kw = dict(q=c.q, out=out, lse=None)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsa.dsa_quant_attention(batch, cache, kw["q"], 0.1, kw["out"], kw["lse"], ws)
    for bad in (dict(sm=0.0), dict(ws=ws[:100]), dict(ws=None)):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_quant_attention(batch, cache, c.q, bad.get("sm", 0.1), out, None,
                                    bad.get("ws", ws))


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("new,far", [(2, False), (60, True)])
def test_outputs_beside_the_cache(code, new, far):
    """One allocation holds workspace, scales, out, keys, lse, values and queries without a
    gap: nothing is refused and nothing outside the outputs is written."""
    c = Case([300, 130], [new, 1], 8, 2, 64, BF16, code, seed=51, far=far)
    want, want_lse = c.run()
    batch = c.batch()
    need = dsa.dsa_quant_attention_workspace_size(batch, c.cache(), c.hq)
    tokens = c.offsets[-1]
    sizes = [-(-need // 16) * 16, c.scales.numel() * 4, want.numel() * 2, c.k.numel(),
             want_lse.numel() * 4, c.v.numel(), c.q.numel() * 2]
    one = torch.full((sum(sizes),), 0x55, dtype=torch.uint8, device=DEV)
    ws, scales, out, k, lse, v, q = one.split(sizes)
    scales = scales.view(torch.float32).view(c.scales.shape)
    k, v = (x.view(code).view(c.k.shape) for x in (k, v))
    q, out = (x.view(BF16).view(c.q.shape) for x in (q, out))
    lse = lse.view(torch.float32).view(want_lse.shape)
    assert out.data_ptr() + tokens * c.hq * 64 * 2 == k.data_ptr()
    scales.copy_(c.scales)
    k.view(torch.uint8).copy_(c.k.view(torch.uint8))
    v.view(torch.uint8).copy_(c.v.view(torch.uint8))
    q.copy_(c.q)
    dsa.dsa_quant_attention(batch, dsa.QuantCache(k, v, scales), q, c.sm_scale, out, lse, ws[:need])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.equal(scales.view(torch.int32), c.scales.view(torch.int32)) and torch.equal(q, c.q)
    assert torch.equal(k.view(torch.uint8), c.k.view(torch.uint8))
    assert torch.equal(v.view(torch.uint8), c.v.view(torch.uint8))


def seen_positions(c):
    """[T]: the positions that each row's token sees."""
    return torch.tensor([max(0, length - n + j + 1) for length, n in zip(c.lens, c.new)
                         for j in range(n)], dtype=torch.float64, device=DEV)


def check_rows(c, out, lse, r=None, beyond=None):
    """As Case.check, with every row held to the positions that it sees itself, whatever the
    longest request has: n of the sums' errors is the row's own.  beyond: what products below
    f16's normal range may be off by, of n positions (2^-37 of the largest scale times code)."""
    r = r or c.reference()
    n = seen_positions(c)[:, None]
    e = (c.d + 9) * 2.0**-23 * r["terms"]
    if beyond is None:
        fine = torch.isfinite(c.scales)
        beyond = 2.0**-37 * float(torch.where(fine, c.scales, 0.0).max()) * 448
    share = 2.0**-11 + 2.0**-16 + n * 2.0**-24 + 2.0**-20 + 2 * e
    tol = torch.finfo(c.dtype).eps / 2 * r["out"].abs() + share[..., None] * r["mean_abs"]
    tol += n[..., None] * beyond + (2.0**-25 if c.dtype == F16 else 0.0)
    err = (out.double() - r["out"]).abs()
    assert (err <= tol).all(), float((err / tol.clamp_min(1e-30)).max())
    empty = torch.isinf(r["lse"])
    assert torch.equal(torch.isneginf(lse), empty)
    off = torch.where(empty, 0.0, (lse.double() - r["lse"]).abs())
    lse_tol = e + 2.0**-16 + n * 2.0**-24 + 2.0**-20 + 2.0**-22 * r["lse"].abs().nan_to_num(0, 0, 0)
    assert (off <= lse_tol).all(), float((off / lse_tol).max())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (64, 49, 1), (128, 8, 2), (128, 33, 1), (256, 8, 2),
                                      (256, 5, 5)])
def test_rows_beside_a_long_request_keep_their_own_accuracy(d, hq, hkv, code, dtype):
    """The tensor core kernel: short requests of one token, of a few and of chunks, beside the
    long one that makes the call large enough."""
    lens = [1, 2, 15, 16, 17, 64, 65, 127, 128, 129, 130, 200, 257, 700, 1500]
    new = [1, 2, 15, 1, 3, 20, 65, 1, 70, 5, 130, 199, 257, 13, 40]
    c = Case(lens, new, hq, hkv, d, dtype, code, seed=60 + hq, far=True)
    check_rows(c, *c.run())


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("d,hq,lens,new", [
    (64, 64, [900, 300], [1, 3]), (128, 40, [900, 700], [1, 1]), (256, 40, [900, 64], [1, 1]),
    (128, 8, [400, 900], [100, 60])])
def test_scales_far_apart_beside_a_long_request(code, d, hq, lens, new):
    """As test_scales_far_apart, rows held to their own lengths."""
    hkv = 1 if hq > 8 else 2
    c = Case(lens, new, hq, hkv, d, F16, code, seed=61, far=True, q_scale=1.0)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    spread_ = torch.randint(-30, 7, c.scales[:, :, 1].shape, generator=g, device=DEV)
    fine = torch.isfinite(c.scales[:, :, 1]) & (c.scales[:, :, 1] > 0)
    c.scales[:, :, 1] = torch.where(fine, torch.exp2(spread_.float() - 7), c.scales[:, :, 1])
    r = c.reference()
    # a product below 2^-26 of the row's largest, which is at most its largest mean_abs
    check_rows(c, *c.run(), r=r, beyond=(2.0**-37 * 448 * r["mean_abs"].amax(-1, keepdim=True)))


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("new", [[2, 1, 3], [0, 0, 0], [60, 1, 33]])
def test_rows_that_no_request_owns_are_not_written(new, far):
    """A step of fixed size: room for 64 tokens a request, offsets that use fewer."""
    lens = [300, 1, 90]
    c = Case(lens, new if max(new) > 12 or not far else [40, 1, 3], 8, 2, 64, BF16, INT8, seed=62,
             far=far)
    tokens, room = c.offsets[-1], 64 * len(c.lens)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    batch = dsa.Batch(i32(c.offsets), i32(c.lens), c.table, c.pages, c.lens, [64] * len(c.lens))
    q = torch.full((room, 8, 64), NAN, dtype=BF16, device=DEV)
    q[:tokens] = c.q
    out, lse = torch.full_like(q, 7.0), torch.full((room, 8), 7.0, device=DEV)
    ws = torch.empty(dsa.dsa_quant_attention_workspace_size(batch, c.cache(), 8), dtype=torch.uint8,
                     device=DEV)
    st = i32([0])
    dsa.dsa_quant_attention(batch, c.cache(), q, c.sm_scale, out, lse, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert (out[tokens:] == 7).all() and (lse[tokens:] == 7).all()
    check_rows(c, out[:tokens], lse[:tokens])


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("d,more", [(64, 0), (128, 0), (256, 0), (64, 40), (128, 40), (256, 40)])
def test_queries_at_the_end_of_bf16(code, d, more):
    """Rows whose largest value is 2^127 or more, alone and beside small ones."""
    c = Case([600, 601, 602] + [500] * (more > 0), [1, 1, 1] + [more] * (more > 0), 4, 2, d, BF16,
             code, seed=63, far=more > 0)
    largest = float(torch.finfo(BF16).max)
    c.q[0] = c.q[0] / c.q[0].abs().amax(-1, keepdim=True) * largest
    c.q[1] = c.q[1] / c.q[1].abs().amax(-1, keepdim=True) * 2.0**126
    c.q[2, :, 5], c.q[2, :, 7] = largest, -(2.0**127)
    c.sm_scale = 2.0**-125
    assert torch.isfinite(c.q).all()
    check_rows(c, *c.run())
