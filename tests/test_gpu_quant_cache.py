"""dsa_quant_append and dsa_quant_read on the GPU against their definitions.

Without turning everything after the 16-bit inputs is one fp32 operation after another, so
scales and codes are compared bit for bit.  With turning, a key differs from its 64-bit
value by e <= 2^-21 of the sum of its two products' sizes; a scale, fp32 quotient of the
largest, by 2^-21 of the block's largest such sum over L (and a rounding, 2^-24); a decoded
key by half a step of its code, e, and the scale's and its reciprocal's roundings
(2^-22 of the value)."""
import random

import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa
from paged_helpers import DEV, PAGE, turn_reference
from quant_helpers import (BLOCK, E4M3, INT8, LARGEST, append_reference, decoded, encode,
                           random_cache, slots_of, tables_of)

pytestmark = pytest.mark.gpu

DEVICE_CHECK = 5
BF16, F16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Append:
    """Requests that bring new tokens to a cache of random codes and scales."""

    def __init__(self, cached, new, hq, hkv, d, dtype, code, seed=0, pad=0):
        g = generator(7000 + seed)
        self.cached, self.new, self.hkv, self.d, self.dtype = cached, new, hkv, d, dtype
        self.lens = [a + b for a, b in zip(cached, new)]
        self.table, self.pages = tables_of(g, self.lens)
        self.slots = slots_of(self.table, cached, new)
        self.slots = torch.cat([self.slots, self.slots.new_full((pad,), -1)])
        tokens = len(self.slots)
        qkv = torch.randn(tokens, hq + 2 * hkv, d, generator=g, device=DEV)
        qkv *= torch.exp(torch.randn(tokens, 1, 1, generator=g, device=DEV))  # scales have to grow
        self.q, self.k, self.v = qkv.to(dtype).split([hq, hkv, hkv], dim=1)
        self.k_pages, self.v_pages, self.scales = random_cache(g, self.pages, hkv, d, code)
        self.q_out = torch.full((tokens, hq, d), NAN, dtype=dtype, device=DEV)

    def run(self, rope=None, positions=None, status=0, **kw):
        cache = dsa.QuantCache(self.k_pages, self.v_pages, self.scales)
        st = i32([0])
        args = dict(q=self.q, k=self.k, v=self.v, q_out=self.q_out, slots=self.slots)
        args.update(kw)
        if self.q.shape[1] == 0:
            args["q"] = args["q_out"] = None
        dsa.dsa_quant_append(cache, rope, positions, args["slots"], args["q"], args["k"],
                             args["v"], args["q_out"], st)
        torch.cuda.synchronize()
        assert int(st.item()) == status

    def reference(self, slots=None):
        slots = self.slots if slots is None else slots
        k, scales, _ = append_reference(self.k_pages, self.scales, 0, slots, self.k.float())
        v, scales, _ = append_reference(self.v_pages, scales, 1, slots, self.v.float())
        return k, v, scales

    def state(self):
        return [x.view(torch.uint8).clone() for x in (self.k_pages, self.v_pages)] + [
            self.scales.clone()]

    def check(self, want):
        for x, y in zip((self.k_pages, self.v_pages), want[:2]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert torch.equal(self.scales, want[2])


@pytest.mark.parametrize("dtype,code", [(BF16, E4M3), (F16, E4M3), (BF16, INT8), (F16, INT8)])
@pytest.mark.parametrize("cached,new,hq,hkv,d,pad", [
    ([0], [1], 1, 1, 64, 0), ([699], [1], 32, 8, 128, 0), ([15, 16, 17, 0], [1, 1, 1, 1], 4, 2, 256, 1),
    ([3, 60, 0], [5, 9, 40], 0, 3, 64, 0), ([37], [300], 8, 2, 128, 3), ([0, 7], [64, 57], 2, 1, 256, 0),
    ([1000 + 3 * b for b in range(90)], [1 + b % 5 for b in range(90)], 8, 4, 128, 2),
    ([31 * b % 50 for b in range(40)], [b * 13 % 70 for b in range(40)], 3, 5, 64, 5)])
def test_append_without_turning_is_exact(dtype, code, cached, new, hq, hkv, d, pad):
    c = Append(cached, new, hq, hkv, d, dtype, code, seed=d + hq, pad=pad)
    want = c.reference()
    c.run()
    c.check(want)
    assert torch.equal(c.q_out, c.q)
    # once more: the same scales and codes
    c.run()
    c.check(want)


@pytest.mark.parametrize("code", [E4M3, INT8])
def test_a_block_written_token_by_token(code):
    """The scale doubles whenever a token does not fit; the older codes follow, and what
    they stand for stays within half a step for each doubling (INT8: half a step of the
    new scale; E4M3: half of the smallest code, the others lose nothing)."""
    c = Append([0], [64], 2, 3, 128, BF16, code, seed=3)
    slots, x = c.slots.clone(), [c.k.clone(), c.v.clone()]
    for t in range(64):
        want = append_reference(c.k_pages, c.scales, 0, slots[t:t + 1], x[0][t:t + 1].float())
        want_v = append_reference(c.v_pages, want[1], 1, slots[t:t + 1], x[1][t:t + 1].float())
        c.run(slots=slots[t:t + 1], q=c.q[t:t + 1], k=x[0][t:t + 1], v=x[1][t:t + 1],
              q_out=c.q_out[t:t + 1])
        c.check((want[0], want_v[0], want_v[1]))
    page, row = slots // PAGE, slots % PAGE
    for which, pool in ((0, c.k_pages), (1, c.v_pages)):
        got = decoded(pool, c.scales, which)[page, :, row]
        scale = c.scales[page, :, which, row // BLOCK].double()[..., None]
        exact = x[which].double()
        if code == INT8:  # at most six halvings of steps: 1/2 + 1/2 + 1/4 ..
            tol = 1.01 * scale
        else:
            tol = 2.0**-4 * exact.abs() + 2.0**-9 * scale
        assert ((got - exact).abs() <= tol + 2.0**-21 * exact.abs()).all()
        top = exact.abs().amax(-1).view(4, BLOCK, 3).amax(1)  # the scale is at most twice need
        need = top / LARGEST[code]
        s = c.scales[page[::BLOCK], :, which, (row // BLOCK)[::BLOCK]].double()
        assert (s >= need * (1 - 2.0**-22)).all()
        first = exact.abs().amax(-1).view(4, BLOCK, 3)[:, 0] / LARGEST[code]
        assert (s <= torch.maximum(2 * need, first) * (1 + 2.0**-22)).all()


@pytest.mark.parametrize("cached,new,hq,hkv,d,dtype,code,sections,interleaved,start", [
    ([0], [1], 1, 1, 64, BF16, E4M3, [32], False, 0),
    ([699], [1], 32, 8, 128, F16, INT8, [64], False, (1 << 20) - 1),
    ([5, 0], [3, 18], 12, 1, 256, BF16, E4M3, [128], False, 1 << 24),
    ([0, 33], [65, 20], 6, 3, 128, F16, INT8, [16, 24, 24], True, 3),
    ([0], [130], 5, 5, 64, BF16, INT8, [8, 0, 8], False, 9),
    ([10, 16], [33, 48], 8, 2, 256, F16, E4M3, [24, 40], True, 77),
    ([0, 1], [3, 2], 0, 2, 128, BF16, E4M3, [32], True, 5),
    ([64] * 20, [7] * 20, 16, 16, 64, F16, E4M3, [5, 7, 4], False, 2**31 - 6000)])
def test_append_with_turning(cached, new, hq, hkv, d, dtype, code, sections, interleaved, start):
    c = Append(cached, new, hq, hkv, d, dtype, code, seed=d + 50, pad=2)
    g = generator(d + hq)
    T, pairs = len(c.slots), sum(sections)
    freq = 10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)
    pos = (start + torch.randint(0, 5000, (len(sections), T), generator=g, device=DEV)).int()
    # fresh scales only: the tokens before in a begun block hold little
    for b, a in enumerate(cached):
        if a % BLOCK:
            page = int(c.table[b, a // PAGE])
            c.scales[page, :, :, a % PAGE // BLOCK] = 2.0**-40
    v_want, v_scales, _ = append_reference(c.v_pages, c.scales, 1, c.slots, c.v.float())
    before = c.state()
    c.run(dsa.Rope(freq, sections, interleaved), pos)
    if hq:
        ref, size = turn_reference(c.q, pos, freq, sections, interleaved)
        small = 2.0**-25 if dtype == F16 else 0.0
        tol = torch.finfo(dtype).eps / 2 * ref.abs() + small + 2.0**-21 * size
        assert ((c.q_out.double() - ref).abs() <= tol).all()
    # values are not turned
    assert torch.equal(c.v_pages.view(torch.uint8), v_want.view(torch.uint8))
    assert torch.equal(c.scales[:, :, 1], v_scales[:, :, 1])
    live = c.slots >= 0
    slots = c.slots[live]
    ref, size = turn_reference(c.k, pos, freq, sections, interleaved)
    ref, size = ref[live], size[live]
    page, row = slots // PAGE, slots % PAGE
    scale = c.scales[page, :, 0, row // BLOCK].double()
    blocks = slots // BLOCK
    for block in blocks.unique().tolist():
        at = blocks == block
        need = ref[at].abs().amax((0, 2)) / LARGEST[code]
        slack = 2.0**-21 * size[at].amax((0, 2)) / LARGEST[code] + 2.0**-23 * need
        s = scale[at][0]
        assert (s >= need - slack).all()
        if int(slots[at][0]) % BLOCK == 0:
            assert (s <= need + slack).all()
        else:
            k = torch.log2(s) + 40
            assert (k == k.round()).all() and (s <= 2 * (need + slack)).all()
    got = decoded(c.k_pages, c.scales, 0)[page, :, row]
    scale = scale[..., None]
    step = scale / 2 if code == INT8 else 2.0**-4 * ref.abs() + 2.0**-10 * scale
    assert ((got - ref).abs() <= step + 2.0**-21 * size * 1.07 + 2.0**-22 * ref.abs()).all()
    # rows of other blocks are as they were
    touched = torch.zeros(c.pages, PAGE, dtype=torch.bool, device=DEV)
    touched[page, row // BLOCK * BLOCK] = True
    touched = touched.view(c.pages, -1, BLOCK)[:, :, :1].expand(-1, -1, BLOCK).reshape(c.pages, PAGE)
    keep = ~touched[:, None, :, None].expand_as(c.k_pages)
    assert torch.equal(c.k_pages.view(torch.uint8)[keep], before[0][keep])


@pytest.mark.parametrize("code", [E4M3, INT8])
def test_infinite_and_nan_values_are_recorded(code):
    c = Append([3], [4], 2, 2, 64, BF16, code, seed=4)
    c.k[1, 0, 5] = INF
    c.k[2, 1, 7] = NAN
    c.v[0, 0, 0] = -INF
    clean = [x.clone() for x in (c.k, c.v)]
    for x in clean:
        x[~torch.isfinite(x)] = 0
    want_k, scales, _ = append_reference(c.k_pages, c.scales, 0, c.slots, clean[0].float())
    want_v, scales, _ = append_reference(c.v_pages, scales, 1, c.slots, clean[1].float())
    c.run(status=DEVICE_CHECK)
    assert torch.equal(c.scales, scales)
    page, row = c.slots // PAGE, c.slots % PAGE
    assert float(c.k_pages[page[1], 0, row[1], 5]) == LARGEST[code]
    assert float(c.v_pages[page[0], 0, row[0], 0]) == -LARGEST[code]
    nan = float(c.k_pages[page[2], 1, row[2], 7])
    assert nan != nan if code == E4M3 else nan == 0
    for got, want, at in ((c.k_pages, want_k, ((1, 0, 5), (2, 1, 7))), (c.v_pages, want_v, ((0, 0, 0),))):
        got, want = got.view(torch.uint8).clone(), want.view(torch.uint8)
        for t, h, i in at:
            got[page[t], h, row[t], i] = want[page[t], h, row[t], i]
        assert torch.equal(got, want)


@pytest.mark.parametrize("code", [E4M3, INT8])
def test_zeros_and_sizes_beyond_the_scales(code):
    """A block of zeros takes the smallest scale and grows out of it; values above L * 2^32
    saturate."""
    c = Append([0, 0, 16], [3, 2, 2], 1, 1, 64, BF16, code, seed=5)
    c.k[:3] = 0
    c.v[3:5] = 2.0**60
    c.v[4, 0, 1] = -(2.0**100)
    want = c.reference()
    c.run()
    c.check(want)
    assert float(c.scales[c.slots[0] // PAGE, 0, 0, 0]) == 2.0**-48
    assert float(c.scales[c.slots[3] // PAGE, 0, 1, 0]) == 2.0**32
    at = c.slots[4:5]
    assert float(c.v_pages[at // PAGE, 0, at % PAGE, 1]) == -LARGEST[code]
    # the next token of the block of zeros
    nxt = c.slots[2:3] + 1
    k, v = torch.randn(2, 1, 1, 64, device=DEV).to(BF16)
    want_k, scales, _ = append_reference(c.k_pages, c.scales, 0, nxt, k.float())
    want_v, scales, _ = append_reference(c.v_pages, scales, 1, nxt, v.float())
    c.run(slots=nxt, q=c.q[:1], k=k, v=v, q_out=c.q_out[:1])
    c.check((want_k, want_v, scales))


@pytest.mark.parametrize("bad", [0.0, -1.0, NAN, INF, 2.0**-60, 2.0**40])
def test_a_begun_block_without_a_scale_is_recorded_and_left(bad):
    c = Append([5, 64], [3, 20], 2, 2, 64, BF16, INT8, seed=6)
    page = int(c.table[0, 0])
    c.scales[page, 1, 0, 0] = bad
    want = c.reference(torch.where(torch.arange(23, device=DEV) < 3, -1, c.slots))
    first = c.reference(torch.where(torch.arange(23, device=DEV) < 3, c.slots, -1))
    c.run(status=DEVICE_CHECK)
    # head 1's keys of the first request's block stay; all else is written
    for got, w, f, old in ((c.k_pages, want[0], first[0], True), (c.v_pages, want[1], first[1], False)):
        for h in range(2):
            for p in range(c.pages):
                src = w if p != page or (h == 1 and old) else f
                assert torch.equal(got[p, h], src[p, h])


def test_slots_out_of_order_or_range_are_recorded_and_skipped():
    c = Append([0], [12], 2, 2, 128, F16, INT8, seed=8)
    base = int(c.slots[0])
    slots = c.slots.clone()
    slots[2] = c.pages * PAGE      # beyond the pool; ends the run of rows 0, 1
    slots[3:] = -1
    want = c.reference(torch.where(torch.arange(12, device=DEV) < 2, slots, -1))
    c.run(status=DEVICE_CHECK, slots=slots)
    c.check(want)
    c = Append([0], [12], 2, 2, 128, F16, INT8, seed=8)
    slots = c.slots.clone()
    slots[5] = base + 2            # a second time: it and nothing else is left out
    keep = slots.clone()
    keep[5] = -1
    want = c.reference(keep)
    c.run(status=DEVICE_CHECK, slots=slots)
    c.check(want)
    c = Append([0], [40], 2, 2, 128, F16, INT8, seed=9)
    slots = c.slots.clone()
    slots[:] = base                # always the same row: the first is kept
    keep = slots.clone()
    keep[1:] = -1
    want = c.reference(keep)
    c.run(status=DEVICE_CHECK, slots=slots)
    c.check(want)


def test_append_in_place_and_from_separate_tensors():
    results = []
    for fused in (True, False):
        c = Append([9], [40], 4, 2, 128, BF16, E4M3, seed=10)
        freq = 10000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float64) / 64)
        pos = torch.arange(40, dtype=torch.int32, device=DEV)
        kw = dict(q_out=c.q) if fused else dict(q=c.q.contiguous(), k=c.k.contiguous(),
                                                v=c.v.contiguous())
        c.run(dsa.Rope(freq), pos, **kw)
        results.append(c.state() + [(c.q if fused else c.q_out).contiguous()])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("dtype,code", [(BF16, E4M3), (F16, E4M3), (BF16, INT8), (F16, INT8)])
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 8), (256, 3)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([700, 64, 65, 3], [700, 64, 65, 3]),
                                      ([300, 17, 90], [5, 0, 90]), ([4, 1000], [7, 100])])
def test_read(dtype, code, d, hkv, lens, new):
    """Whole requests, their last tokens, and more tokens than there is context: those rows,
    and the rows behind the last token, stay."""
    g = generator(d + len(lens))
    table, pages = tables_of(g, lens)
    k, v, scales = random_cache(g, pages, hkv, d, code)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    T = offsets[-1]
    wide = torch.full((T + 2, 2 * hkv + 1, d), 7.0, dtype=dtype, device=DEV)
    want = wide.clone()
    for b, (length, n) in enumerate(zip(lens, new)):
        for j in range(n):
            p = length - n + j
            if p >= 0:
                page, row = table[b, p // PAGE].long(), p % PAGE
                for which, x in ((0, k), (1, v)):
                    # fp32 product, rounded once
                    y = x[page, :, row].float() * scales[page, :, which, row // BLOCK][..., None]
                    want[offsets[b] + j, which * hkv:(which + 1) * hkv] = y.to(dtype)
    batch = dsa.Batch(i32(offsets), i32(lens), table, pages, lens, new)
    cache, st = dsa.QuantCache(k, v, scales), i32([0])
    dsa.dsa_quant_read(batch, cache, wide[:, :hkv], wide[:, hkv:2 * hkv], st)
    assert torch.equal(wide, want) and int(st.item()) == 0
    for which in (0, 1):  # one of the two
        one = torch.full((T, hkv, d), 7.0, dtype=dtype, device=DEV)
        dsa.dsa_quant_read(batch, cache, *((one, None) if which == 0 else (None, one)))
        assert torch.equal(one, want[:T, which * hkv:(which + 1) * hkv])


def test_read_records_bad_pages_and_requests():
    g = generator(77)
    lens = [200, 100, 70]
    table, pages = tables_of(g, lens)
    k, v, scales = random_cache(g, pages, 2, 64, INT8)
    cache, T = dsa.QuantCache(k, v, scales), sum(lens)
    offsets = [0, 200, 300, 370]

    def read(table, seq_lens, status):
        out = torch.full((T, 2, 64), 7.0, dtype=BF16, device=DEV)
        st = i32([0])
        dsa.dsa_quant_read(dsa.Batch(i32(offsets), i32(seq_lens), table, pages, lens, lens), cache,
                           out, None, st)
        assert int(st.item()) == status
        return out
    want = read(table, lens, 0)
    bad = table.clone()
    bad[0, 1], bad[1, 0] = pages, -3
    out = read(bad, lens, DEVICE_CHECK)
    skipped = torch.zeros(T, dtype=torch.bool, device=DEV)
    skipped[64:128] = skipped[200:264] = True
    assert (out[skipped] == 7).all() and torch.equal(out[~skipped], want[~skipped])
    out = read(table, [200, 1 << 20, 70], DEVICE_CHECK)
    skipped[:] = False
    skipped[200:300] = True
    assert (out[skipped] == 7).all() and torch.equal(out[~skipped], want[~skipped])


def test_scales_outside_their_range_count_as_its_ends():
    g = generator(78)
    table, pages = tables_of(g, [64])
    k, v, scales = random_cache(g, pages, 1, 64, INT8)
    page = int(table[0, 0])
    scales[page, 0, 0] = torch.tensor([0.0, NAN, -3.0, INF], device=DEV)
    out = torch.empty(64, 1, 64, dtype=BF16, device=DEV)
    dsa.dsa_quant_read(dsa.Batch(i32([0, 64]), i32([64]), table, pages, [64], [64]),
                       dsa.QuantCache(k, v, scales), out, None)
    ends = torch.tensor([2.0**-48] * 3 + [2.0**33], device=DEV).repeat_interleave(16)
    assert torch.equal(out[:, 0], (k[page, 0].float() * ends[:, None]).to(BF16))


def test_a_pool_beyond_32_bit_offsets():
    """More than 2^32 bytes of codes and 2^31 of elements, the last pages in use."""
    c = Append([5, 40], [30, 90], 2, 8, 128, BF16, E4M3, seed=11)
    want = c.reference()
    n = c.pages
    pages = (1 << 32) // (8 * PAGE * 128) + 50
    big = [torch.empty(pages, 8, PAGE, 128, dtype=E4M3, device=DEV) for _ in range(2)]
    scales = torch.empty(pages, 8, 2, 4, dtype=torch.float32, device=DEV)
    for x, y in zip(big + [scales], (c.k_pages, c.v_pages, c.scales)):
        x[pages - n:] = y
    c.k_pages, c.v_pages, c.scales = *big, scales
    c.run(slots=torch.where(c.slots >= 0, c.slots + (pages - n) * PAGE, -1))
    batch = dsa.Batch(i32([0, 35, 165]), i32(c.lens), c.table + (pages - n), pages, c.lens, c.lens)
    out = torch.empty(165, 8, 128, dtype=BF16, device=DEV)
    dsa.dsa_quant_read(batch, dsa.QuantCache(*big, scales), out, None)
    c.k_pages, c.v_pages, c.scales = (x[pages - n:] for x in (*big, scales))
    c.check(want)
    ref = decoded(want[0], want[2], 0)
    rows = torch.cat([slots_of(c.table, [0], [n]) if b == 0 else slots_of(c.table[1:], [0], [n])
                      for b, n in enumerate(c.lens)])
    assert torch.equal(out, ref[rows // PAGE, :, rows % PAGE].float().to(BF16))


def test_on_another_stream_and_in_a_graph():
    c = Append([9, 64], [40, 1], 4, 2, 128, BF16, INT8, seed=12)
    start = c.state()
    want = c.reference()
    cache = dsa.QuantCache(c.k_pages, c.v_pages, c.scales)
    batch = dsa.Batch(i32([0, 49, 114]), i32(c.lens), c.table, c.pages, c.lens, c.lens)
    out = torch.zeros(114, 2, 128, dtype=BF16, device=DEV)

    def reset():
        c.k_pages.view(torch.uint8).copy_(start[0])
        c.v_pages.view(torch.uint8).copy_(start[1])
        c.scales.copy_(start[2])
        out.zero_()

    def calls(stream=None):
        dsa.dsa_quant_append(cache, None, None, c.slots, c.q, c.k, c.v, c.q_out, stream=stream)
        dsa.dsa_quant_read(batch, cache, out, None, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    s.synchronize()
    c.check(want)
    read = out.clone()
    graph = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        c.check(want)
        assert torch.equal(out, read)


def test_python_checks():
    c = Append([0], [6], 4, 2, 64, BF16, E4M3, seed=13)
    cache = dsa.QuantCache(c.k_pages, c.v_pages, c.scales)
    pos = torch.zeros(1, 6, dtype=torch.int32, device=DEV)
    rope = dsa.Rope(torch.ones(32, dtype=torch.float64, device=DEV))
    for bad in (dict(q=c.q[:3]), dict(k=c.k[..., ::2]), dict(k=c.k.transpose(1, 2)),
                dict(v=c.v.float()), dict(slots=c.slots[:5]), dict(slots=c.slots.int()),
                dict(positions=pos.view(-1)[:5]), dict(q=c.q.cpu())):
        kw = dict(positions=pos, slots=c.slots, q=c.q, k=c.k, v=c.v, q_out=c.q_out)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsa.dsa_quant_append(cache, rope, **kw)
    for k, v, s in ((c.k_pages[:, :, :32], c.v_pages[:, :, :32], c.scales),
                    (c.k_pages, c.v_pages[:1], c.scales), (c.k_pages, c.v_pages, c.scales[:, :, :1]),
                    (c.k_pages.float(), c.v_pages.float(), c.scales),
                    (c.k_pages, c.v_pages, c.scales.half()), (c.k_pages, c.v_pages.view(INT8), c.scales)):
        with pytest.raises((TypeError, ValueError)):
            dsa.QuantCache(k, v, s)
    batch = dsa.Batch(i32([0, 6]), i32([6]), c.table, c.pages, [6], [6])
    out = torch.empty(6, 2, 64, dtype=BF16, device=DEV)
    for k, v in ((out[:5], None), (out.float(), None), (out, out.half()), (out[..., ::2], None),
                 (None, None), (out.view(6, 1, 128), None)):
        with pytest.raises((TypeError, ValueError)):
            dsa.dsa_quant_read(batch, cache, k, v)
    assert encode(torch.tensor([0.5]), INT8).item() == 0  # the oracle's ties go to even


def pieces(c, *parts):
    """(slots, k, v): tokens of c, None for one that is not stored, in the order given."""
    at = [t for part in parts for t in part]
    pick = torch.tensor([0 if t is None else t for t in at], device=DEV)
    gone = torch.tensor([t is None for t in at], device=DEV)
    return torch.where(gone, -1, c.slots[pick]), c.k[pick], c.v[pick]


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("gap", [1, 3, 14, 15, 16, 31, 40, 200, 1000])
@pytest.mark.parametrize("cached,more,beyond", [(0, 0, False), (0, 0, True), (5, 0, False), (0, 700, False)])
def test_a_block_again_behind_tokens_that_are_not_stored_is_left_and_recorded(cached, gap, code,
                                                                               more, beyond):
    """Four tokens of a block, tokens that are not stored, four more of the block and the
    first three of the next: the second four are left out, and nothing else is."""
    c = Append([cached, 0], [11 + 16 - 8 - cached, more], 2, 3, 64, BF16, code, seed=20)
    first, later = list(range(0, 4)), list(range(4, 8))
    fresh = [t for t in range(len(c.slots) - more) if (cached + t) // BLOCK == 1][:3]
    tail = list(range(len(c.slots) - more, len(c.slots)))
    slots, k, v = pieces(c, first, [None] * gap, later, fresh, tail)
    if beyond:
        slots[4:4 + gap] = c.pages * PAGE + 3
    keep = slots.clone()
    keep[4 + gap:8 + gap] = -1
    keep[4:4 + gap] = -1
    want_k, scales, _ = append_reference(c.k_pages, c.scales, 0, keep, k.float())
    want_v, scales, _ = append_reference(c.v_pages, scales, 1, keep, v.float())
    q = torch.zeros(len(slots), 2, 64, dtype=BF16, device=DEV)
    c.run(status=DEVICE_CHECK, slots=slots, q=q, k=k, v=v, q_out=torch.empty_like(q))
    c.check((want_k, want_v, scales))


def test_other_blocks_behind_tokens_that_are_not_stored_are_written():
    """A gap before another block, before the first token and after the last one."""
    c = Append([0, 3], [40, 60], 2, 2, 128, F16, INT8, seed=21)
    slots, k, v = pieces(c, [None] * 5, list(range(0, 16)), [None] * 45, list(range(16, 40)),
                         [None], list(range(40, 100)), [None] * 7)
    want_k, scales, _ = append_reference(c.k_pages, c.scales, 0, slots, k.float())
    want_v, scales, _ = append_reference(c.v_pages, scales, 1, slots, v.float())
    q = torch.zeros(len(slots), 2, 128, dtype=F16, device=DEV)
    c.run(slots=slots, q=q, k=k, v=v, q_out=torch.empty_like(q))
    c.check((want_k, want_v, scales))


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("before", [0, 1, 7, 500])
@pytest.mark.parametrize("rows,kept", [
    ([0, 5, 3, 5, 6], [1, 1, 0, 0, 1]), ([2, 9, 1, 2, 3, 9, 10, 4], [1, 1, 0, 0, 0, 0, 1, 0]),
    ([0, 15, 1, 2, 3, 14, 15], [1, 1, 0, 0, 0, 0, 0]),
    (list(range(16)) + [0, 1, 2], [1] * 16 + [0] * 3),
    ([0] * 15 + [1, 2, 3], [1] + [0] * 14 + [1, 0, 0])])
def test_slots_of_a_block_that_do_not_exceed_those_before_are_left_out(rows, kept, before, code):
    """No row is written twice: a token counts where its slot exceeds every earlier one of the
    block, and is among the block's first sixteen tokens."""
    n = len(rows)
    c = Append([0, 0], [32, max(before, 1)], 2, 2, 128, F16, code, seed=23)
    start = int(c.slots[0]) // PAGE * PAGE
    slots = torch.cat([c.slots[32:32 + before],
                       torch.tensor([start + r for r in rows], device=DEV), c.slots[16:20]])
    k, v = (x[torch.arange(len(slots), device=DEV) % len(c.slots)] for x in (c.k, c.v))
    k[before + 2:before + n] *= 3  # a token that is left out does not count for the scale
    keep = slots.clone()
    keep[before:before + n] = torch.where(torch.tensor(kept, device=DEV) > 0,
                                          slots[before:before + n], -1)
    want_k, scales, _ = append_reference(c.k_pages, c.scales, 0, keep, k.float())
    want_v, scales, _ = append_reference(c.v_pages, scales, 1, keep, v.float())
    q = torch.zeros(len(slots), 2, 128, dtype=F16, device=DEV)
    c.run(status=DEVICE_CHECK, slots=slots, q=q, k=k, v=v, q_out=torch.empty_like(q))
    c.check((want_k, want_v, scales))


def test_layouts_of_one_buffer():
    """Queries, keys, values and turned queries anywhere in one buffer, a few rows of them at
    strides that agree or not: refused exactly where q_out shares an element with an input
    that it is not, else written as from separate tensors."""
    rng, d, seen = random.Random(3), 64, [0, 0]
    freq = 10000.0 ** (-torch.arange(32, device=DEV, dtype=torch.float64) / 32)
    for _ in range(400):
        tokens, hq, hkv = rng.randint(1, 5), rng.randint(1, 3), rng.randint(1, 2)
        common = (hq + 2 * hkv) * d + rng.choice([0, 8, 200])

        def layout(heads):
            stride = common if rng.random() < 0.7 else heads * d + 8 * rng.randint(0, 60)
            return heads, 8 * rng.randint(0, 200), stride
        parts = [layout(hq), layout(hkv), layout(hkv), layout(hq)]
        if rng.random() < 0.5:  # as in a fused projection, here and there
            parts = [(h, at, common) for h, at in ((hq, 0), (hkv, hq * d), (hkv, (hq + hkv) * d),
                                                   (hq, rng.choice([0, 0, 8, tokens * common])))]
        size = max(at + (tokens - 1) * s + h * d for h, at, s in parts)
        buffer = torch.randn(size, device=DEV).to(BF16)
        q, k, v, out = (torch.as_strided(buffer, (tokens, h, d), (s, d, 1), at) for h, at, s in parts)
        own = [{at + t * s + i for t in range(tokens) for i in range(h * d)} for h, at, s in parts]
        in_place = parts[0][1] == parts[3][1] and (tokens == 1 or parts[0][2] == parts[3][2])
        clash = bool(own[3] & (own[1] | own[2])) or (not in_place and bool(own[3] & own[0]))
        c = Append([3], [tokens], 1, hkv, d, BF16, INT8, seed=30)
        pos = torch.arange(tokens, dtype=torch.int32, device=DEV) + 1000
        start, before = c.state(), buffer.clone()
        want = torch.empty(tokens, hq, d, dtype=BF16, device=DEV)
        c.run(dsa.Rope(freq), pos, q=q.clone(), k=k.clone(), v=v.clone(), q_out=want)
        state = c.state()
        for x, y in zip((c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.scales), start):
            x.copy_(y)
        seen[clash] += 1
        if clash:
            with pytest.raises(dsa.DsaError):
                c.run(dsa.Rope(freq), pos, q=q, k=k, v=v, q_out=out)
            torch.cuda.synchronize()
            assert torch.equal(buffer, before)
        else:
            c.run(dsa.Rope(freq), pos, q=q, k=k, v=v, q_out=out)
            c.check(state)
            assert torch.equal(out, want)
            torch.as_strided(before, out.shape, out.stride(), parts[3][1]).copy_(want)
            assert torch.equal(buffer, before)
    assert min(seen) > 50, seen


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("tokens", [1, 9])
def test_outputs_beside_and_between_the_arrays(code, tokens):
    """Read: one allocation holds keys' codes, k_out, the scales, v_out and the values' codes
    without a gap, and k_out and v_out as slices of the same rows do not overlap.  Append: q_out
    in the place of k_out, of a stride that leaves the scales between two rows of it."""
    hkv, d = 2, 64
    c = Append([30 - tokens], [tokens], 2, hkv, d, BF16, code, seed=31)
    want = c.reference()
    lens, row = [30], hkv * d * 2
    batch = dsa.Batch(i32([0, tokens]), i32(lens), c.table, c.pages, lens, [tokens])
    sizes = [c.k_pages.numel(), tokens * row, c.scales.numel() * 4, tokens * row, c.v_pages.numel()]
    one = torch.full((sum(sizes),), 0x55, dtype=torch.uint8, device=DEV)
    k, k_out, scales, v_out, v = one.split(sizes)
    k, v = (x.view(code).view(c.k_pages.shape) for x in (k, v))
    scales = scales.view(torch.float32).view(c.scales.shape)
    for x, y in ((k, c.k_pages), (v, c.v_pages)):
        x.view(torch.uint8).copy_(y.view(torch.uint8))
    scales.copy_(c.scales)
    k_out, v_out = (x.view(BF16).view(tokens, hkv, d) for x in (k_out, v_out))
    cache, st = dsa.QuantCache(k, v, scales), i32([0])
    dsa.dsa_quant_append(cache, None, None, c.slots, c.q, c.k, c.v, k_out, st)
    assert torch.equal(k_out, c.q)
    dsa.dsa_quant_read(batch, cache, k_out, v_out, st)
    wide = torch.zeros(tokens, 2 * hkv, d, dtype=BF16, device=DEV)
    dsa.dsa_quant_read(batch, cache, wide[:, :hkv], wide[:, hkv:], st)
    assert int(st.item()) == 0
    assert torch.equal(k_out, wide[:, :hkv]) and torch.equal(v_out, wide[:, hkv:])
    ref = decoded(want[0], want[2], 0)[c.slots // PAGE, :, c.slots % PAGE]
    assert torch.equal(k_out, ref.float().to(BF16))
    c.k_pages, c.v_pages, c.scales = k, v, scales
    c.check(want)
    # rows of queries on both sides of an array of scales
    if tokens > 1:
        apart = c.scales.numel() * 2 + hkv * d  # values from row to row: 1 KB and more
        buffer = torch.full((apart * tokens,), 7.0, dtype=BF16, device=DEV)
        between = buffer[hkv * d:apart].view(torch.float32).view(c.scales.shape)
        between.copy_(c.scales)
        out = torch.as_strided(buffer, (tokens, 2, d), (apart, d, 1), 0)
        dsa.dsa_quant_append(dsa.QuantCache(k, v, between), None, None, c.slots, c.q, c.k, c.v, out, st)
        assert torch.equal(out, c.q) and torch.equal(between, c.scales) and int(st.item()) == 0


@pytest.mark.parametrize("new", [[3, 5, 0], [0, 0, 0], [40, 1, 9], [64, 64, 64]])
def test_a_step_of_fixed_size_with_unused_rows(new):
    """Tables, append and read of a captured step with room for 64 tokens a request: rows that
    no request fills are left as they are, and nothing is recorded."""
    cached, hkv, d, room = [10, 0, 70], 2, 64, 192
    c = Append(cached, new, 2, hkv, d, BF16, INT8, seed=40)
    cache, st = dsa.QuantCache(c.k_pages, c.v_pages, c.scales), i32([0])
    lens = [a + b for a, b in zip(cached, new)]
    table = torch.full((3, 8), -7, dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.table
    held = [-(-n // PAGE) for n in cached]
    free = [int(table[b, i]) for b in range(3) for i in range(held[b], -(-lens[b] // PAGE))]
    offsets, seq = i32([0] * 4), i32([0] * 3)
    slots = torch.empty(room, dtype=torch.int64, device=DEV)
    positions, taken = torch.empty(room, dtype=torch.int32, device=DEV), i32([0])
    tokens = sum(new)
    q, k, v = (torch.zeros(room, h, d, dtype=BF16, device=DEV) for h in (2, hkv, hkv))
    q[:tokens], k[:tokens], v[:tokens] = c.q, c.k, c.v
    q_out, k_out, v_out = torch.full((3, room, hkv, d), 7.0, dtype=BF16, device=DEV)
    want = c.reference()
    free = i32(free + [c.pages - 1])  # one more than is needed
    dsa.dsa_build_tables(i32(cached), i32(new), free, c.pages, table, offsets, seq, slots, positions,
                         None, taken, st)
    dsa.dsa_quant_append(cache, None, None, slots, q, k, v, q_out, st)
    batch = dsa.Batch(offsets, seq, table, c.pages, [8 * PAGE] * 3, [64] * 3)
    assert batch.total_q == room
    dsa.dsa_quant_read(batch, cache, k_out, v_out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    c.check(want)
    assert (k_out[tokens:] == 7).all() and (v_out[tokens:] == 7).all()
    page, row = c.slots // PAGE, c.slots % PAGE
    for out, pool, which in ((k_out, want[0], 0), (v_out, want[1], 1)):
        assert torch.equal(out[:tokens], decoded(pool, want[2], which)[page, :, row].float().to(BF16))


@pytest.mark.parametrize("offsets", [[0, 5, 9, 7], [0, -4, 3, 9], [2, 3, 4, 5], [0, 3, 4, 40]])
def test_offsets_that_contradict_the_host_sizes_are_still_recorded(offsets):
    g = generator(79)
    lens = [20, 30, 40]
    table, pages = tables_of(g, lens)
    k, v, scales = random_cache(g, pages, 1, 64, E4M3)
    out, st = torch.full((12, 1, 64), 7.0, dtype=BF16, device=DEV), i32([0])
    batch = dsa.Batch(i32([0, 4, 8, 12]), i32(lens), table, pages, lens, [4, 4, 4])
    batch.q_offsets.copy_(i32(offsets))
    dsa.dsa_quant_read(batch, dsa.QuantCache(k, v, scales), out, None, st)
    assert int(st.item()) == DEVICE_CHECK


@pytest.mark.parametrize("dtype,code,hq,hkv,d", [(BF16, E4M3, 4, 2, 128), (F16, INT8, 2, 1, 64),
                                                 (BF16, INT8, 1, 1, 256)])
@pytest.mark.parametrize("cached,new,pad", [
    ([37], [456], 0), ([37], [457], 0), ([0, 9], [400, 190], 3), ([5], [912], 0), ([13], [913], 1),
    ([6], [1824], 0), ([0, 30], [1000, 829], 1), ([7], [3000], 0), ([2 * b for b in range(300)],
                                                                    [1 + b % 4 for b in range(300)], 7)])
def test_appends_of_every_number_of_tokens_to_a_cta(dtype, code, hq, hkv, d, cached, new, pad):
    """Calls of 457, 913 and 1825 tokens and more give a CTA two, four and eight."""
    c = Append(cached, new, hq, hkv, d, dtype, code, seed=d + hq, pad=pad)
    want = fast_reference(c)
    c.run()
    c.check(want)
    assert torch.equal(c.q_out, c.q)


def fast_reference(c):
    """append_reference for many tokens: all blocks at once, in the same fp32 operations."""
    t = torch.nonzero(c.slots >= 0)[:, 0]
    slots = c.slots[t]
    blocks, nth = torch.unique_consecutive(slots // BLOCK, return_inverse=True)
    page, part = blocks // (PAGE // BLOCK), blocks % (PAGE // BLOCK)
    fresh = torch.zeros(len(blocks), device=DEV).index_reduce_(
        0, nth, (slots % BLOCK == 0).float(), "amax")[:, None] > 0
    pools, scales = [], c.scales.clone()
    for which, pool, x in ((0, c.k_pages, c.k), (1, c.v_pages, c.v)):
        pool, x = pool.clone(), x[t].float()
        top = torch.zeros(len(blocks), c.hkv, device=DEV).index_reduce_(0, nth, x.abs().amax(-1), "amax")
        need = (top / torch.full_like(top, LARGEST[pool.dtype])).clamp(2.0**-48, 2.0**32)
        begun = scales[page, :, which, part]
        k = torch.zeros_like(begun, dtype=torch.int32)
        for _ in range(100):
            k += (torch.ldexp(begun, k) < need).int()
        k = torch.where(fresh, 0, k)
        scale = torch.where(fresh, need, torch.ldexp(begun, k))
        scales[page, :, which, part] = scale
        rows = pool.view(torch.uint8).view(-1, c.hkv, PAGE // BLOCK, BLOCK, c.d)
        held = rows[page, :, part].view(pool.dtype).float()
        rows[page, :, part] = encode(torch.ldexp(held, -k[..., None, None]), pool.dtype).view(torch.uint8)
        rows[page[nth], :, part[nth], slots % BLOCK] = encode(
            x * (torch.ones_like(scale) / scale)[nth][..., None], pool.dtype).view(torch.uint8)
        pools.append(pool)
    return (*pools, scales)


@pytest.mark.parametrize("dtype,code,interleaved", [(BF16, INT8, False), (F16, E4M3, True)])
def test_a_long_prompt(dtype, code, interleaved):
    """Sixteen tokens to a CTA, from 16384 on; turned, and the same prompt in calls of at most
    2000 tokens that end at blocks' borders gives the same cache and queries, bit for bit."""
    c = Append([11], [16384 + 5 + 3], 2, 1, 64, dtype, code, seed=33, pad=2)
    want = fast_reference(c)
    start = c.state()
    c.run()
    c.check(want)
    freq = 10000.0 ** (-torch.arange(32, device=DEV, dtype=torch.float64) / 32)
    pos = torch.arange(len(c.slots), dtype=torch.int32, device=DEV) + 11
    results = []
    for each in (len(c.slots), 2000):
        for x, y in zip((c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.scales), start):
            x.copy_(y)
        c.q_out.fill_(NAN)
        at = 0
        while at < len(c.slots):
            to = min(len(c.slots), at + each - (0 if at or each > 2000 else 11))  # 11 are cached
            part = slice(at, to)
            c.run(dsa.Rope(freq, interleaved=interleaved), pos[part], slots=c.slots[part], q=c.q[part],
                  k=c.k[part], v=c.v[part], q_out=c.q_out[part])
            at = to
        results.append(c.state() + [c.q_out.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("requests", [31, 32, 33, 64, 65, 100, 700, 1025, 3000])
@pytest.mark.parametrize("some_empty", [False, True])
def test_reads_of_many_requests(requests, some_empty):
    """More requests than are looked through at a time, among them such that bring nothing."""
    g, rng = generator(requests), random.Random(requests)
    lens = [rng.randint(1, 90) for _ in range(requests)]
    new = [0 if some_empty and rng.random() < 0.6 else rng.randint(0, min(n, 20)) for n in lens]
    new[-1] = max(new[-1], 1)
    table, pages = tables_of(g, lens)
    k, v, scales = random_cache(g, pages, 1, 64, INT8)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    owner = torch.repeat_interleave(torch.arange(requests), torch.tensor(new))
    at = torch.arange(offsets[-1]) - torch.tensor(offsets)[owner]
    pos = (torch.tensor(lens) - torch.tensor(new))[owner] + at
    page, row = table[owner.to(DEV), (pos // PAGE).to(DEV)].long(), (pos % PAGE).to(DEV)
    out, st = torch.full((2, offsets[-1], 1, 64), 7.0, dtype=F16, device=DEV), i32([0])
    batch = dsa.Batch(i32(offsets), i32(lens), table, pages, lens, new)
    dsa.dsa_quant_read(batch, dsa.QuantCache(k, v, scales), out[0], out[1], st)
    assert int(st.item()) == 0
    for which, x in ((0, k), (1, v)):
        want = x[page, :, row].float() * scales[page, :, which, row // BLOCK][..., None]
        assert torch.equal(out[which], want.to(F16))


@pytest.mark.parametrize("gap", [2046, 2047, 2048, 2049, 4097, 20000])
@pytest.mark.parametrize("again", [False, True])
def test_a_block_behind_thousands_of_tokens_that_are_not_stored(gap, again):
    """The same look back over more slots than a CTA sees at a time, to the block itself and to
    another one."""
    c = Append([0], [40], 2, 2, 64, BF16, INT8, seed=24)
    slots, k, v = pieces(c, list(range(0, 4)), [None] * gap,
                         list(range(4, 8)) if again else list(range(20, 24)), list(range(32, 35)))
    keep = slots.clone()
    if again:
        keep[4 + gap:8 + gap] = -1
    want_k, scales, _ = append_reference(c.k_pages, c.scales, 0, keep, k.float())
    want_v, scales, _ = append_reference(c.v_pages, scales, 1, keep, v.float())
    q = torch.zeros(len(slots), 2, 64, dtype=BF16, device=DEV)
    c.run(status=DEVICE_CHECK if again else 0, slots=slots, q=q, k=k, v=v, q_out=torch.empty_like(q))
    c.check((want_k, want_v, scales))
