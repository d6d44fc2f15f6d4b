"""dsa_paged_attention where values, scores, batches and buffers are out of the ordinary.

Tolerances are those of test_gpu_paged_attention, but for probabilities rounded to f16,
which are held at 2^15 times their size: half a step (eps / 2) of those from 2^-29 of the
row's largest on, and half of f16's smallest step, 2^-40, of those below."""
import copy

import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa
from test_gpu_paged_attention import BF16, DEV, F16, FP8, NAN, Case

pytestmark = pytest.mark.gpu

INF = float("inf")


def tolerances(c, r):
    """(of out, of lse) for the reference r of case c."""
    n = max(c.lens)
    bf16_p = c.k.dtype == BF16
    e = (c.d + 8) * 2.0**-23 * r["terms"]
    tol = (torch.finfo(c.dtype).eps / 2 * r["out"].abs() +
           torch.finfo(BF16 if bf16_p else F16).eps / 2 * r["mean_abs"] +
           (2 * e + n * 2.0**-24 + 2.0**-20)[..., None] * r["mean_abs"])
    if not bf16_p:
        tol += n * 2.0**-40 * r["max_abs"][..., None]
    if c.dtype == F16:
        tol += 2.0**-25
    fine = torch.where(torch.isinf(r["lse"]), 0.0, r["lse"])
    return tol, e + n * 2.0**-24 + 2.0**-20 + 2.0**-22 * fine.abs()


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


@pytest.mark.parametrize("dtype,kv", [(F16, F16), (BF16, FP8), (F16, FP8), (BF16, BF16)])
@pytest.mark.parametrize("requests,length,d", [
    (1, 700, 128),     # a cluster to the unit
    (200, 300, 64),    # half-size CTAs
    (160, 2048, 64), (160, 2048, 128), (160, 1100, 256)])  # the list
def test_many_small_probabilities_beside_a_large_one(requests, length, d, dtype, kv):
    """A position about 18 above all others, whose value is 0: what is left of the
    output is the sum of the others' probabilities, some 2^-26 each."""
    c = Case([length] * requests, [1] * requests, 4, 1, d, dtype, kv, seed=41)
    k, v = c.k.float(), c.v.float() + 4 / c.scales[1]
    k = torch.where(k.isnan(), k, 0.0)
    first = c.table[:, 0].long()
    k[first, :, 5] = 18.0 / d**0.5 / c.scales[0]
    v[first, :, 5] = 0.0
    c.k, c.v = k.to(kv), v.to(kv)
    c.q[:] = 1.0
    out, lse = c.run()
    r = c.reference()
    tol, lse_tol = tolerances(c, r)
    err = (out.double() - r["out"]).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse.double() - r["lse"]).abs() <= lse_tol).all()


@pytest.mark.parametrize("dtype,kv", [(F16, F16), (F16, FP8), (BF16, FP8)])
def test_scores_of_millions(dtype, kv):
    """Scores whose steps in fp32 are of the order of 1: the largest stays a finite
    probability.  Each row sees one position far above the rest."""
    c = Case([300, 700], [1, 1], 4, 2, 64, dtype, kv, seed=42)
    k = torch.where(c.k.float().isnan(), NAN, 0.0)
    for b, length in enumerate(c.lens):
        at = length - 7
        k[c.table[b, at // 64].long(), :, at % 64] = 448.0
    c.k = k.to(kv)
    c.q[:] = 448.0 + 64 * torch.arange(4, device=DEV)[:, None]
    c.sm_scale = 1.37 / (c.scales[0])
    out, _ = c.run()
    for b, length in enumerate(c.lens):
        at = length - 7
        want = c.v[c.table[b, at // 64].long(), :, at % 64].float() * c.scales[1]
        want = want.repeat_interleave(2, dim=0)
        assert ((out[b].float() - want).abs() <= torch.finfo(dtype).eps * want.abs()).all()


@pytest.mark.parametrize("lens,new,hq,hkv", [
    ([200, 130, 67], [5, 3, 4], 8, 2),                       # clusters
    ([200, 130, 67] * 60, [5, 3, 4] * 60, 8, 2),             # half-size CTAs, or the list
    ([2900, 1300, 64, 700] * 12, [5, 2, 4, 1] * 12, 16, 4),  # the list
    ([150, 90], [150, 60], 6, 2)])                           # a prompt
@pytest.mark.parametrize("d,dtype,kv,bad", [
    (64, BF16, BF16, NAN), (128, BF16, BF16, INF), (256, BF16, BF16, -INF), (64, F16, F16, -INF),
    (128, F16, F16, NAN), (256, F16, F16, INF), (64, BF16, FP8, NAN), (128, F16, FP8, NAN),
    (256, BF16, FP8, NAN)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(lens, new, hq, hkv, d, dtype, kv,
                                                                 bad):
    """The last two new tokens' values (the last, of two; none, of one) are not finite in
    two dims of each head.  Rows before them are as if they were not there."""
    c = Case(lens, new, hq, hkv, d, dtype, kv, seed=43)
    r = c.reference()
    tol, lse_tol = tolerances(c, r)
    want = r["out"].clone()
    g = hq // hkv
    v = c.v.float()
    for b, (length, n) in enumerate(zip(lens, new)):
        for at in range(max(length - 2, length - n + 1), length):
            page = c.table[b, at // 64].long()
            for h in range(hkv):
                dims = [(5 * b + h) % d, (7 * h + at) % d]
                v[page, h, at % 64, dims] = bad
                first = c.offsets[b] + at - (length - n)  # the first row that sees it
                for dim in dims:
                    want[first:c.offsets[b + 1], h * g:(h + 1) * g, dim] = bad
    c.v = v.to(kv)
    out, lse = c.run()
    out = out.double()
    assert torch.equal(out.isnan(), want.isnan())
    same = torch.isfinite(want)
    assert torch.equal(torch.where(same | want.isnan(), 0.0, out),
                       torch.where(same | want.isnan(), 0.0, want))
    err = torch.where(same, out - want, 0.0).abs()
    assert (err <= tol).all(), float((err / tol.clamp_min(1e-30)).max())
    assert ((lse.double() - r["lse"]).abs() <= lse_tol).all()


@pytest.mark.parametrize("kv", [BF16, FP8])
@pytest.mark.parametrize("copies", [1, 90])
def test_rows_that_see_nothing_are_zero_whatever_the_values(kv, copies):
    """More new tokens than context, and values of the context that are not numbers."""
    lens, new = [3, 2, 70] * copies, [6, 5, 2] * copies
    c = Case(lens, new, 8, 2, 128, BF16, kv, seed=44)
    v = c.v.float()
    for b in range(len(lens)):
        v[c.table[b, 0].long(), :, :3] = NAN
    c.v = v.to(kv)
    out, lse = c.run()
    for b, (length, n) in enumerate(zip(lens, new)):
        blind = slice(c.offsets[b], c.offsets[b] + max(0, n - length))
        assert (out[blind] == 0).all() and torch.isneginf(lse[blind]).all()
        seeing = slice(blind.stop, c.offsets[b + 1])
        assert out[seeing].isnan().all() and torch.isfinite(lse[seeing]).all()


def test_scale_factors_below_fp32s_range():
    """bf16 queries of 2^-60 over FP8 keys under sm_scale 2^-100: all scores are 0, and
    positions past a row's view stay masked."""
    c = Case([200, 90], [3, 1], 4, 2, 64, BF16, FP8, seed=45)
    c.q *= 2.0**-60
    c.sm_scale = 2.0**-100
    out, lse = c.run()
    c.check(out, lse)


def test_buffers_of_another_shape_are_refused():
    c = Case([300, 64], [1, 1], 4, 2, 64, BF16, seed=46)
    batch, cache = c.batch(), c.cache()
    ws = torch.empty(dsa.dsa_paged_attention_workspace_size(batch, cache, 4), dtype=torch.uint8,
                     device=DEV)

    def empty(*shape, dtype=BF16):
        return torch.zeros(*shape, dtype=dtype, device=DEV)
    want, want_lse = c.run()
    for out, lse in ((empty(2, 4, 64), empty(2, 4, dtype=torch.float32)),
                     (empty(5, 4, 64), empty(5, 4, dtype=torch.float32)),      # a larger capacity
                     (empty(2, 256), empty(8, dtype=torch.float32)),           # heads flattened
                     (empty(600), empty(11, dtype=torch.float32))):            # flat
        dsa.dsa_paged_attention(batch, cache, c.q, c.sm_scale, out, lse, ws)
        assert torch.equal(out.view(-1)[:512], want.view(-1))
        assert torch.equal(lse.view(-1)[:8], want_lse.view(-1))
    for out, lse in ((empty(2, 64, 4), None), (empty(4, 2, 64), None), (empty(2, 8, 64), None),
                     (empty(2, 512), None),
                     (empty(2, 4, 64), empty(4, 2, dtype=torch.float32)),
                     (empty(2, 4, 64), empty(2, 8, dtype=torch.float32))):
        with pytest.raises(ValueError):
            dsa.dsa_paged_attention(batch, cache, c.q, c.sm_scale, out, lse, ws)


@pytest.mark.parametrize("axes", [2, 3])
def test_positions_of_another_shape_are_refused(axes):
    """Axes are as far apart as there are tokens: of a wider buffer the second would be
    read in the wrong place."""
    tokens, sections = 6, [8] * axes
    qkv = torch.randn(tokens, 8, 64, device=DEV).to(BF16)
    q, k, v = qkv.split([4, 2, 2], dim=1)
    pool = torch.zeros(2, 3, 2, 64, 64, dtype=BF16, device=DEV)
    freq = torch.rand(8 * axes, dtype=torch.float64, device=DEV)
    cache, rope = dsa.KvCache(pool[0], pool[1]), dsa.Rope(freq, sections)
    slots = torch.arange(tokens, device=DEV)
    out = torch.empty(tokens, 4, 64, dtype=BF16, device=DEV)
    pos = torch.randint(0, 1000, (axes, 9), dtype=torch.int32, device=DEV)

    def call(p):
        dsa.dsa_rope_append(cache, rope, p, slots, q, k, v, out)
        return out.clone()
    for bad in (pos, pos.T.contiguous()[:tokens], pos[:, :tokens].T.contiguous(),
                pos[:axes - 1, :tokens].contiguous()):
        with pytest.raises(ValueError):
            call(bad)
    live = pos[:, :tokens].contiguous()
    want = call(live)
    more = torch.cat([live, live[:1]])  # axes that the heads do not use
    for good in (live.view(-1), more, more.view(-1)):
        assert torch.equal(call(good), want)
    # one axis: the first of a larger buffer
    rope = dsa.Rope(freq[:8])
    want = call(live[:1])
    assert torch.equal(call(pos[0]), want) and torch.equal(call(pos[:1]), want)
