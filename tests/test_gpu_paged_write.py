"""dsa_build_tables and dsa_rope_append on the GPU against plain references.

Tolerance of the turned values: one rounding to the output type, half a step
(eps / 2 of the value; for E4M3 2^-4, and half of its smallest step 2^-9), plus
fp32 arithmetic: the fraction of a turn in fp32 (2^-25 of at most pi), a cosine
and a sine of 2 ulp each and three roundings, together below 8 * 2^-24 of
|x| + |y|, the sizes of the pair's two products."""
import random

import numpy as np
import pytest
import torch

import dsa_sparse_attention_step_gb300 as dsa
from paged_helpers import (DEV, E4M3_MAX, PAGE, ceil_pages, tables_reference, turn_reference)

pytestmark = pytest.mark.gpu

DEVICE_CHECK = 5


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run_tables(cached, new, free, num_pages, table, cap, stream=None):
    n = len(cached)
    out = dict(table=i32(table.tolist()).reshape(n, -1),
               q_offsets=torch.full((n + 1,), -7, dtype=torch.int32, device=DEV),
               seq_lens=torch.full((n,), -7, dtype=torch.int32, device=DEV),
               slots=torch.full((cap,), -7, dtype=torch.int64, device=DEV),
               positions=torch.full((cap,), -7, dtype=torch.int32, device=DEV),
               requests=torch.full((cap,), -7, dtype=torch.int32, device=DEV),
               taken=i32([-7]), status=i32([0]))
    dsa.dsa_build_tables(i32(cached), i32(new), i32(free), num_pages, out["table"],
                         out["q_offsets"], out["seq_lens"], out["slots"], out["positions"],
                         out["requests"], out["taken"], out["status"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_tables(cached, new, free, num_pages, table, cap):
    got = run_tables(cached, new, free, num_pages, table, cap)
    ref = tables_reference(cached, new, free, num_pages, table, cap)
    for name, want in zip(("table", "q_offsets", "seq_lens", "slots", "positions", "requests"), ref):
        assert np.array_equal(got[name], want), name
    assert int(got["taken"][0]) == ref[6]
    assert int(got["status"][0]) == (0 if ref[7] else DEVICE_CHECK)


def step(rng, cached, new, spare=2, extra_width=1):
    """Free list, pool size and block table for the given lengths."""
    held = [ceil_pages(max(c, 0)) for c in cached]
    grown = [ceil_pages(max(c, 0) + max(n, 0)) - h for c, n, h in zip(cached, new, held)]
    total = sum(held) + sum(grown) + spare
    ids = list(range(total))
    rng.shuffle(ids)
    table = np.full((len(cached), max(1, max(h + g for h, g in zip(held, grown)) + extra_width)),
                    -9, dtype=np.int64)
    for b, h in enumerate(held):
        table[b, :h] = [ids.pop() for _ in range(h)]
    return ids, total, table


@pytest.mark.parametrize("requests,cached,new", [
    (1, 0, 1), (1, 63, 1), (1, 64, 1), (1, 0, 64), (1, 0, 65), (1, 127, 2), (3, 200, 0),
    (5, 0, 4099), (37, 1000, 7), (512, 90, 1), (513, 200, 3), (4096, 130, 2), (4095, 0, 9)])
def test_tables(requests, cached, new):
    rng = random.Random(requests * 31 + cached + new)
    c = [rng.randint(0, cached) for _ in range(requests)]
    n = [rng.randint(0, new) for _ in range(requests)]
    c[0], n[0] = cached, new
    free, total, table = step(rng, c, n)
    check_tables(c, n, free, total, table, sum(n))
    check_tables(c, n, free, total, table, sum(n) + 130)  # unused rows at the end


def test_tables_without_new_tokens():
    rng = random.Random(1)
    c, n = [0, 64, 5], [0, 0, 0]
    free, total, table = step(rng, c, n)
    check_tables(c, n, free, total, table, 0)
    check_tables(c, n, free, total, table, 5)


def test_tables_report_what_does_not_fit():
    rng = random.Random(2)
    c, n = [10, 100, 64, 0], [60, 5, 64, 300]
    free, total, table = step(rng, c, n)
    check_tables(c, n, free[:3], total, table, sum(n))             # free list too short
    check_tables(c, n, [], total, table, sum(n))                   # empty free list
    check_tables(c, n, [total + 5] + free[1:], total, table, sum(n))  # page ids outside the pool
    check_tables(c, n, [-3] + free[1:], total, table, sum(n))
    bad = table.copy()
    bad[1, 1] = total                                              # the open page of a request
    check_tables(c, n, free, total, bad, sum(n))
    check_tables(c, n, free, total, table[:, :2], sum(n))          # more pages than a row holds
    check_tables([10, -1, 64, 0], n, free, total, table, sum(n))   # negative lengths
    check_tables(c, [60, -5, 64, 300], free, total, table, sum(n))
    check_tables(c, n, free, total, table, sum(n) - 200)           # too many tokens
    check_tables(c, n, free, total, table, 61)


def test_tables_lengths_whose_sums_pass_32_bits():
    """Three requests of 2^30 cached tokens and as many new ones do not fit the
    table; the fourth is unaffected but for the offset, which stops at the cap."""
    big = 1 << 30
    table = np.full((4, 3), 1, dtype=np.int64)
    got = run_tables([big] * 3 + [5], [big] * 3 + [7], [2, 3], 8, table, 100)
    assert got["q_offsets"].tolist() == [0, 100, 100, 100, 100]
    assert got["seq_lens"].tolist() == [2**31 - 1] * 3 + [12]
    assert np.array_equal(got["table"], table) and int(got["taken"][0]) == 0
    assert (got["slots"] == -1).all() and int(got["status"][0]) == DEVICE_CHECK


def test_tables_only_offsets():
    n = [3, 0, 70]
    table = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    q, s, t = i32([0] * 4), i32([0] * 3), i32([0])
    dsa.dsa_build_tables(i32([1, 2, 3]), i32(n), i32([5, 6, 7]), 9, table, q, s, pages_taken=t)
    assert q.tolist() == [0, 3, 3, 73] and s.tolist() == [4, 2, 73] and t.tolist() == [1]
    assert table.tolist() == [[0] * 4, [0] * 4, [0, 5, 0, 0]]


def rope_case(seed, T, hq, hkv, d, dtype, fp8, sections, interleaved, start=0, fused=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    heads = hq + 2 * hkv
    qkv = torch.randn(T, heads, d, generator=g, device=DEV).to(dtype)
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pages = ceil_pages(T) + 3
    ids = torch.randperm(pages * PAGE, generator=g, device=DEV)[:T].to(torch.int64)
    store = torch.float8_e4m3fn if fp8 else dtype
    pool = torch.randn(2, pages, hkv, PAGE, d, generator=g, device=DEV).to(store)
    pairs = sum(sections)
    freq = 10000.0 ** (-torch.arange(max(pairs, 1), device=DEV, dtype=torch.float64)[:pairs] / max(pairs, 1))
    pos = start + torch.randint(0, 5000, (max(len(sections), 1), T), generator=g, device=DEV)
    return q, k, v, pool, ids, freq, pos.to(torch.int32)


def half_step(ref, dtype):
    small = 2.0**-25 if dtype == torch.float16 else 0.0
    return torch.finfo(dtype).eps / 2 * ref.abs() + small


@pytest.mark.parametrize("T,hq,hkv,d,dtype,fp8,sections,interleaved,start", [
    (1, 1, 1, 64, torch.bfloat16, False, [32], False, 0),
    (1, 32, 8, 128, torch.float16, False, [64], False, (1 << 20) - 1),
    (7, 12, 1, 256, torch.bfloat16, True, [128], False, 1 << 24),
    (65, 6, 3, 128, torch.float16, True, [16, 24, 24], True, 3),
    (130, 5, 5, 64, torch.bfloat16, False, [8, 0, 8], False, 9),
    (33, 8, 2, 256, torch.float16, False, [24, 40], True, 77),
    (3, 0, 2, 128, torch.bfloat16, True, [32], True, 5),
    (5, 4, 2, 128, torch.bfloat16, False, [], False, 0),
    (301, 16, 16, 64, torch.float16, True, [5, 7, 4], False, 2**31 - 6000)])
def test_rope_append(T, hq, hkv, d, dtype, fp8, sections, interleaved, start):
    q, k, v, pool, slots, freq, pos = rope_case(T + d, T, hq, hkv, d, dtype, fp8, sections,
                                                interleaved, start)
    ks, vs = (0.02, 0.05) if fp8 else (1.0, 1.0)
    drop = [0, T // 2] if T > 4 else []
    slots[drop] = -1
    before = pool.clone()
    cache = dsa.KvCache(pool[0], pool[1], ks, vs)
    rope = dsa.Rope(freq, sections, interleaved)
    q_out = torch.zeros(T, hq, d, dtype=dtype, device=DEV)
    st = i32([0])
    dsa.dsa_rope_append(cache, rope, pos, slots, q if hq else None, k, v, q_out if hq else None, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    keep = [i for i in range(T) if i not in drop]
    page, row = slots[keep] // PAGE, slots[keep] % PAGE
    if hq:
        ref, size = turn_reference(q, pos, freq, sections, interleaved)
        assert ((q_out.double() - ref).abs() <= half_step(ref, dtype) + 2.0**-21 * size).all()
    kref, size = turn_reference(k, pos, freq, sections, interleaved)
    for x, ref, size, scale in ((pool[0], kref, size, ks), (pool[1], v.double(), v.double().abs(), vs)):
        got, ref, size = x[page, :, row].double(), ref[keep], size[keep]
        if fp8:
            ref, size = (ref / scale).clamp(-E4M3_MAX, E4M3_MAX), size / scale
            tol = 2.0**-4 * ref.abs() + 2.0**-10 + 2.0**-21 * size
        else:
            tol = half_step(ref, dtype) + 2.0**-21 * size
        assert ((got - ref).abs() <= tol).all()
    # nothing else in the pools changed
    for new, old in zip(pool, before):
        new, old = new.view(torch.uint8), old.view(torch.uint8)
        new[page, :, row] = old[page, :, row]
        assert torch.equal(new, old)


def test_rope_append_in_place_and_from_separate_tensors():
    args = (9, 33, 4, 2, 128, torch.bfloat16, False, [64], False, 10)
    outs = []
    for fused in (True, False):
        q, k, v, pool, slots, freq, pos = rope_case(*args, fused=fused)
        dst = q if fused else torch.empty_like(q)
        dsa.dsa_rope_append(dsa.KvCache(pool[0], pool[1]), dsa.Rope(freq), pos, slots, q, k, v, dst)
        outs.append((dst.contiguous(), pool))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_rope_append_values_beyond_fp8_saturate_and_nan_stays():
    q, k, v, pool, slots, freq, pos = rope_case(3, 4, 2, 1, 64, torch.bfloat16, True, [32], False)
    v[0, 0, :4] = torch.tensor([1e30, -1e30, float("nan"), float("inf")])
    out = torch.empty(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    dsa.dsa_rope_append(dsa.KvCache(pool[0], pool[1], 0.1, 0.1), dsa.Rope(freq), pos, slots, q, k, v,
                        out)
    got = pool[1][slots[0] // PAGE, 0, slots[0] % PAGE, :4].float().tolist()
    assert got[0] == 448 and got[1] == -448 and got[2] != got[2] and got[3] == 448


def test_rope_append_slots_beyond_the_pool_are_reported_and_skipped():
    q, k, v, pool, slots, freq, pos = rope_case(4, 6, 2, 2, 128, torch.float16, False, [64], False)
    want = pool.clone()
    slots[2] = pool.shape[1] * PAGE
    slots[4] = 2**40
    keep = [0, 1, 3, 5]
    st = i32([0])
    out = torch.empty(6, 2, 128, dtype=torch.float16, device=DEV)
    cache = dsa.KvCache(pool[0], pool[1])
    dsa.dsa_rope_append(cache, dsa.Rope(freq), pos, slots, q, k, v, out, st)
    assert int(st.item()) == DEVICE_CHECK
    s = slots[keep]
    assert torch.equal(pool[1][s // PAGE, :, s % PAGE], v[keep])
    for x, old in zip(pool, want):
        x[s // PAGE, :, s % PAGE] = old[s // PAGE, :, s % PAGE]
    assert torch.equal(pool, want)


def test_python_checks_of_shapes_and_types():
    q, k, v, pool, slots, freq, pos = rope_case(5, 6, 4, 2, 64, torch.bfloat16, False, [32], False)
    cache, rope, out = dsa.KvCache(pool[0], pool[1]), dsa.Rope(freq), torch.empty_like(q)
    for bad in (dict(q=q[:3]), dict(k=k[..., ::2]), dict(k=k.transpose(1, 2)), dict(v=v.float()),
                dict(slots=slots[:5]), dict(slots=slots.int()), dict(positions=pos.view(-1)[:5]),
                dict(q=q.cpu())):
        kw = dict(positions=pos, slots=slots, q=q, k=k, v=v, q_out=out)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsa.dsa_rope_append(cache, rope, **kw)
    with pytest.raises(ValueError):
        dsa.Rope(freq, [16, 15])
    with pytest.raises(ValueError):
        dsa.KvCache(pool[0][:, :, :32], pool[1][:, :, :32])
    with pytest.raises(dsa.DsaError):  # a 16-bit cache holds the type of the queries
        dsa.dsa_rope_append(cache, rope, pos, slots, q.half(), k.half(), v.half(), out.half())
