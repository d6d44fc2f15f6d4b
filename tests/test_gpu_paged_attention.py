"""dsa_paged_attention on the GPU against the definition in 64 bits.

Tolerances, per output value, from the arithmetic alone:
  - the output's rounding: half a step, eps / 2 of the value;
  - P rounded to the operand type (bf16 for a bf16 cache, else f16): half a step
    of every probability, eps / 2 of sum p |v|; f16 steps below 2^-14 are 2^-24, so
    at most 2^-25 |v| per position where p is counted from the row's maximum 1;
  - a score's error e: fp32 dot products of D terms, (D + 8) 2^-23 of the sum of
    the terms' sizes (this also covers bf16 queries scaled into f16); it moves p
    by e, and out by 2 e sum p |v|;
  - fp32 sums over n positions and exponentials: n 2^-24 + 2^-20 of sum p |v|."""
import random

import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa
from paged_helpers import DEV, PAGE, attention_reference, ceil_pages

pytestmark = pytest.mark.gpu

DEVICE_CHECK, TIMEOUT = 5, 6
BF16, F16, FP8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
NAN = float("nan")


class Case:
    """A batch over shuffled pages; cache rows past a context's end and pages
    that no request holds are NaN."""

    def __init__(self, lens, new, hq, hkv, d, dtype=BF16, kv=None, seed=0, q_scale=2.0, width=None):
        kv = kv or dtype
        g = torch.Generator(device=DEV)
        g.manual_seed(1000 + seed)
        self.lens, self.new, self.hq, self.d, self.dtype = list(lens), list(new), hq, d, dtype
        counts = [ceil_pages(n) for n in lens]
        self.pages = sum(counts) + 3
        order = torch.randperm(self.pages, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((len(lens), width or max(1, max(counts))), -5, dtype=torch.int32,
                                device=DEV)
        pools = torch.randn(2, self.pages, hkv, PAGE, d, generator=g, device=DEV)
        used = 0
        for b, c in enumerate(counts):
            ids = order[used:used + c]
            self.table[b, :c] = ids
            used += c
            if lens[b] % PAGE:
                pools[:, ids[-1].long(), :, lens[b] % PAGE:] = NAN
        pools[:, order[used:].long()] = NAN
        self.scales = (0.02, 0.04) if kv == FP8 else (1.0, 1.0)
        if kv == FP8:
            pools = pools / torch.tensor(self.scales, device=DEV).view(2, 1, 1, 1, 1)
        self.k, self.v = (x.to(kv) for x in pools)
        self.offsets = [0]
        for n in new:
            self.offsets.append(self.offsets[-1] + n)
        self.q = (q_scale * torch.randn(self.offsets[-1], hq, d, generator=g, device=DEV)).to(dtype)
        self.sm_scale = d ** -0.5

    def cache(self):
        return dsa.KvCache(self.k, self.v, *self.scales)

    def batch(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        return dsa.Batch(i32(self.offsets), i32(self.lens), self.table, self.pages, self.lens,
                         self.new)

    def run(self, q=None, status=0, batch=None):
        batch, cache = batch or self.batch(), self.cache()
        out = torch.full(self.q.shape, NAN, dtype=self.dtype, device=DEV)
        lse = torch.full(self.q.shape[:2], NAN, dtype=torch.float32, device=DEV)
        need = dsa.dsa_paged_attention_workspace_size(batch, cache, self.hq)
        ws = torch.full((need // 4 + (1 << 20),), NAN, dtype=torch.float32, device=DEV)  # any contents
        ws[(need + 3) // 4:] = 7.0  # not part of it
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        dsa.dsa_paged_attention(batch, cache, self.q if q is None else q, self.sm_scale, out, lse,
                                ws, st)
        torch.cuda.synchronize()
        assert int(st.item()) == status
        assert (ws[(need + 3) // 4:] == 7.0).all()
        return out, lse

    def reference(self):
        return attention_reference(self.q, self.k, self.v, *self.scales, self.sm_scale,
                                   self.offsets, self.lens, self.table, self.pages)

    def check(self, out, lse):
        r = self.reference()
        n = max(self.lens)
        p_type = BF16 if self.k.dtype == BF16 else F16
        e = (self.d + 8) * 2.0**-23 * r["terms"]
        tol = (torch.finfo(self.dtype).eps / 2 * r["out"].abs() +
               torch.finfo(p_type).eps / 2 * r["mean_abs"] +
               (2 * e + n * 2.0**-24 + 2.0**-20)[..., None] * r["mean_abs"])
        if p_type == F16:
            tol += n * 2.0**-25 * r["max_abs"][..., None]
        if self.dtype == F16:
            tol += 2.0**-25
        err = (out.double() - r["out"]).abs()
        assert (err <= tol).all(), float((err / tol.clamp_min(1e-30)).max())
        empty = torch.isinf(r["lse"])
        assert torch.equal(torch.isneginf(lse), empty)
        fine = torch.where(empty, 0.0, r["lse"])
        off = (torch.where(empty, 0.0, lse.double()) - fine).abs()
        assert (off <= e + n * 2.0**-24 + 2.0**-20 + 2.0**-22 * fine.abs()).all()


def spread(seed, requests, top):
    rng = random.Random(seed)
    return [rng.randint(1, top) for _ in range(requests - 1)] + [top]


@pytest.mark.parametrize("dtype,kv", [(BF16, BF16), (F16, F16), (BF16, FP8), (F16, FP8)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,new", [(1, 1, 1), (8, 8, 1), (12, 1, 1), (32, 8, 5), (40, 2, 1),
                                        (8, 1, 9), (15, 3, 27)])
@pytest.mark.parametrize("filler,top", [(0, 1500), (170, 2100), (170, 300)])
def test_formats_and_head_layouts(dtype, kv, d, hq, hkv, new, filler, top):
    """Few requests (a cluster to each KV head), and more than there are SMs, most of
    one token (equal shares of one list; for short contexts a CTA to a KV head)."""
    lens = [max(n, new) for n in spread(d + hq, 5, top)] + [1] * filler
    c = Case(lens, [new] * 5 + [1] * filler, hq, hkv, d, dtype, kv, seed=hq)
    c.check(*c.run())


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191,
                                    192, 193, 257])
@pytest.mark.parametrize("new,kv", [(1, BF16), (7, FP8)])
def test_lengths(length, new, kv):
    c = Case([length, 3 * length], [min(new, length), 1], 4, 2, 128, BF16, kv, seed=length)
    c.check(*c.run())
    for d in (64, 256):
        c = Case([length, 3 * length] * 45, [min(new, length), 1] * 45, 4, 2, d, BF16, kv, seed=length)
        c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,d,length,new", [(4, 1, 128, 70001, 1), (3, 3, 64, 33333, 3),
                                                 (12, 1, 256, 20011, 4), (8, 1, 256, 60011, 5),
                                                 (16, 1, 256, 60013, 2), (16, 1, 256, 60017, 4),
                                                 (24, 1, 128, 60019, 1), (48, 1, 128, 60021, 1),
                                                 (64, 1, 64, 60023, 1), (40, 1, 64, 60025, 1)])
def test_one_long_request_is_split_and_joined(hq, hkv, d, length, new):
    c = Case([length], [new], hq, hkv, d, BF16, seed=length)
    c.check(*c.run())


def test_many_ragged_requests():
    rng = random.Random(5)
    lens = [rng.choice([1, 5, 64, 130, 700, 2900]) for _ in range(700)]
    new = [min(rng.choice([0, 1, 1, 2, 3]), n) for n in lens]
    c = Case(lens, new, 8, 2, 64, F16, seed=4)
    c.check(*c.run())


def test_a_prompt_over_many_row_tiles():
    c = Case([333, 200, 90], [333, 60, 1], 6, 2, 128, BF16, seed=8)
    c.check(*c.run())


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_rows_that_see_nothing(kv):
    """Padding requests (no context), and tokens before position 0."""
    c = Case([0, 100, 0, 3, 2], [1, 2, 5, 6, 3], 8, 2, 128, BF16, kv, seed=2)
    out, lse = c.run()
    c.check(out, lse)
    for rows in (slice(0, 1), slice(3, 8), slice(8, 11), slice(14, 15)):
        assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()
    c = Case([0, 0], [1, 1], 4, 4, 64, BF16, kv)
    out, lse = c.run()
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_requests_without_new_tokens_write_nothing():
    c = Case([500, 64, 1, 90], [0, 1, 0, 0], 4, 2, 64, F16, seed=3)
    c.check(*c.run())


def test_scores_far_apart_and_equal():
    """One position dominating, late and early, and all scores equal."""
    c = Case([900, 900, 900], [1, 1, 1], 4, 1, 128, BF16, seed=6, q_scale=60.0)
    c.q[2] = 0
    c.check(*c.run())


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_a_row_of_nan_stays_alone(kv):
    c = Case([300, 90], [3, 1], 8, 2, 128, BF16, kv, seed=21)
    want, want_lse = c.run()
    c.q[1, 2, 5] = NAN
    out, lse = c.run()
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
    out[1, 2], lse[1, 2] = want[1, 2], want_lse[1, 2]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_queries_of_extreme_size_over_fp8():
    """bf16 queries beyond f16's range, and far below it."""
    c = Case([600, 601, 602], [1, 1, 1], 4, 2, 64, BF16, FP8, seed=7)
    c.q[0] *= 2.0**20
    c.q[1] *= 2.0**-30
    c.q[2, :, ::2] *= 2.0**-20
    c.sm_scale = 2.0**-22
    c.check(*c.run())


def test_pages_outside_the_pool_are_left_out_and_reported():
    c = Case([700, 300], [1, 2], 8, 2, 128, BF16, seed=9)
    for b, i, page in ((0, 0, -1), (0, 7, c.pages), (1, 4, 1 << 30)):
        c.table[b, i] = page
    out, lse = c.run(status=DEVICE_CHECK)
    c.check(out, lse)
    c.table[1] = -1  # nothing left to see
    out, lse = c.run(status=DEVICE_CHECK)
    c.check(out, lse)


def test_requests_that_contradict_the_host_sizes_are_reported_and_not_written():
    c = Case([200, 300, 64], [1, 1, 1], 4, 2, 64, BF16, seed=10)
    b = c.batch()
    b.seq_lens[1] = 1 << 20
    out, lse = c.run(status=DEVICE_CHECK, batch=b)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    ok, _ = c.run()
    assert torch.equal(out[[0, 2]], ok[[0, 2]])
    b = c.batch()
    b.q_offsets[3] = 7
    out, _ = c.run(status=DEVICE_CHECK, batch=b)
    assert torch.isnan(out[2]).all() and torch.equal(out[:2], ok[:2])


@pytest.mark.parametrize("requests", [6, 400])
def test_offsets_that_run_back_and_forth_are_reported(requests):
    """Every second request ends before it begins; the others share their rows.
    What the rows then hold is anybody's, but nothing else is touched."""
    c = Case([200] * requests, [0] * requests, 4, 2, 64, BF16, seed=20)
    c.new = [3] + [0] * (requests - 1)
    c.offsets = [0] + [3, 0] * (requests // 2)
    c.q = torch.randn(3, 4, 64, device=DEV).to(BF16)
    out, lse = c.run(status=DEVICE_CHECK)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_queries_as_a_slice_of_a_projection():
    c = Case([130, 700], [2, 1], 8, 2, 128, BF16, seed=11)
    wide = torch.full((3, 12, 128), NAN, dtype=BF16, device=DEV)
    wide[:, 2:10] = c.q
    out, lse = c.run(q=wide[:, 2:10])
    same, _ = c.run()
    assert torch.equal(out, same)


def test_results_do_not_change_from_run_to_run():
    c = Case(spread(3, 40, 5000), [1] * 40, 16, 2, 128, BF16, FP8, seed=12)
    first = c.run()
    for _ in range(3):
        again = c.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("hq,hkv,d,new,kv", [(32, 8, 128, 1, BF16), (16, 4, 128, 6, FP8),
                                             (8, 8, 64, 1, BF16), (8, 4, 256, 1, BF16)])
def test_calls_in_a_row_over_a_long_cache(hq, hkv, d, new, kv):
    """Copies from HBM that finish out of order, passes that follow one another
    without a wait, the workspace shared."""
    c = Case([150000, 99000], [new] * 2, hq, hkv, d, BF16, kv, seed=18)
    want, want_lse = c.run()
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, cache, hq), dtype=torch.uint8,
                     device=DEV)
    outs = [(torch.zeros_like(want), torch.zeros_like(want_lse)) for _ in range(12)]
    for out, lse in outs:
        dsa.dsa_paged_attention(batch, cache, c.q, c.sm_scale, out, lse, ws)
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    c.check(want, want_lse)


def test_batch_invariant_switch():
    """Under the switch a request's results do not depend on its batch."""
    lens, new = [5000, 77, 1300], [1, 2, 5]
    c = Case(lens, new, 8, 2, 128, BF16, seed=13)
    prev = dsa.dsa_set_batch_invariant(True)
    try:
        out, lse = c.run()
        c.check(out, lse)
        for b in range(3):
            alone = Case(lens, new, 8, 2, 128, BF16, seed=13)
            rows = slice(c.offsets[b], c.offsets[b + 1])
            alone.lens, alone.new, alone.offsets = [lens[b]], [new[b]], [0, new[b]]
            alone.table, alone.q = alone.table[b:b + 1].contiguous(), alone.q[rows].contiguous()
            o, l = alone.run()
            assert torch.equal(o, out[rows]) and torch.equal(l, lse[rows])
    finally:
        dsa.dsa_set_batch_invariant(prev)


def test_on_another_stream_and_in_a_graph():
    c = Case([3000, 650], [1, 3], 8, 2, 128, BF16, seed=14)
    want, want_lse = c.run()
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, cache, 8), dtype=torch.uint8,
                     device=DEV)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsa.dsa_paged_attention(batch, cache, c.q, c.sm_scale, out, lse, ws, None, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_paged_attention(batch, cache, c.q, c.sm_scale, out, lse, ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_pool_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements, its last pages in use."""
    c = Case([1000], [2], 8, 8, 128, BF16, seed=15)
    pages = (1 << 31) // (8 * PAGE * 128) + 40
    pool = torch.empty(pages, 8, PAGE, 128, dtype=BF16, device=DEV)
    n = c.k.shape[0]
    pool[pages - n:] = c.k
    c.table += pages - n
    c.k = c.v = pool
    c.pages = pages
    out, lse = c.run()
    del pool
    low = Case([1000], [2], 8, 8, 128, BF16, seed=15)
    low.v = low.k
    want, want_lse = low.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("lens,hkv,d,kv", [
    ([900, 300], 2, 128, BF16),           # clusters
    ([300] * 90, 2, 64, FP8),             # half-size CTAs, four copying warps
    ([30000, 700, 64], 2, 128, BF16)])    # the list and its joining kernel
def test_a_wait_that_runs_out_is_reported_and_the_stream_recovers(lens, hkv, d, kv):
    c = Case(lens, [1] * len(lens), 4 * hkv, hkv, d, BF16, kv, seed=22)
    want, want_lse = c.run()
    batch, cache, out = c.batch(), c.cache(), torch.empty_like(want)
    ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, cache, c.hq),
                     dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsa.dsa_test_paged_attention_wait_timeout(batch, cache, c.q, c.sm_scale, out, None, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == TIMEOUT
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_no_lse_and_no_tokens():
    c = Case([300], [1], 4, 2, 64, BF16, seed=16)
    want, _ = c.run()
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, cache, 4), dtype=torch.uint8,
                     device=DEV)
    out = torch.zeros_like(want)
    dsa.dsa_paged_attention(batch, cache, c.q, c.sm_scale, out, None, ws)
    assert torch.equal(out, want)


def test_python_checks():
    c = Case([300, 64], [1, 1], 4, 2, 64, BF16, seed=17)
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, cache, 4), dtype=torch.uint8,
                     device=DEV)
    out = torch.empty_like(c.q)
    for bad in (dict(q=c.q[:1]), dict(q=c.q.float()), dict(q=c.q[..., ::2]), dict(out=out[:1]),
                dict(out=out.half()), dict(lse=torch.empty(3, device=DEV))):
        kw = dict(q=c.q, out=out, lse=None)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsa.dsa_paged_attention(batch, cache, kw["q"], 0.1, kw["out"], kw["lse"], ws)
    for bad in (dict(sm=0.0), dict(ws=ws[:100]), dict(ws=None)):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_paged_attention(batch, cache, c.q, bad.get("sm", 0.1), out, None,
                                    bad.get("ws", ws))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_at_the_end_of_bf16_over_fp8(d):
    """Rows whose largest value is 2^127 or more, alone and beside small ones."""
    c = Case([600, 601, 602], [1, 1, 1], 4, 2, d, BF16, FP8, seed=63)
    largest = float(torch.finfo(BF16).max)
    c.q[0] = c.q[0] / c.q[0].abs().amax(-1, keepdim=True) * largest
    c.q[1] = c.q[1] / c.q[1].abs().amax(-1, keepdim=True) * 2.0**126
    c.q[2, :, 5], c.q[2, :, 7] = largest, -(2.0**127)
    c.sm_scale = 2.0**-119  # times 0.02 log2 e the least that is taken
    c.k = (c.k.float() * 2.0**-6).to(FP8)
    assert torch.isfinite(c.q).all()
    c.check(*c.run())
