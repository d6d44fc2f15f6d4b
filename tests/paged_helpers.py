"""Plain references of the paged key/value operators, in Python and 64 bits,
written from the definitions in include/dsa.h."""
import numpy as np
import torch

PAGE = 64
DEV = "cuda:0"
E4M3_MAX = 448.0


def ceil_pages(n):
    return -(-n // PAGE)


def tables_reference(cached, new, free, num_pages, table, max_tokens):
    """(table, q_offsets, seq_lens, slots, positions, requests, taken, ok)."""
    table = table.copy()
    ok, taken = True, 0
    offsets, lens = [0], []
    slots, positions, requests = [], [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        fits = c >= 0 and n >= 0 and ceil_pages(max(c, 0) + max(n, 0)) <= table.shape[1]
        ok &= fits
        c, n = max(c, 0), max(n, 0)
        lens.append(min(c + n, 2**31 - 1))
        if fits:
            for lp in range(ceil_pages(c), ceil_pages(c + n)):
                page = int(free[taken]) if taken < len(free) else -1
                taken += 1
                if not 0 <= page < num_pages:
                    page, ok = -1, False
                table[b, lp] = page
        room = max_tokens - offsets[-1]
        ok &= n <= room
        for j in range(min(n, room)):
            page = int(table[b, (c + j) // PAGE]) if fits else -1
            if fits and not 0 <= page < num_pages:
                page, ok = -1, False
            slots.append(page * PAGE + (c + j) % PAGE if page >= 0 else -1)
            positions.append(c + j)
            requests.append(b)
        offsets.append(offsets[-1] + min(n, room))
    rest = max_tokens - len(slots)
    return (table, np.array(offsets), np.array(lens), np.array(slots + [-1] * rest),
            np.array(positions + [0] * rest), np.array(requests + [-1] * rest), taken, ok)


def turn_reference(x, positions, inv_freq, sections, interleaved):
    """float64 [T, H, D] turned, and for each value the sum of the absolute
    values of its two products."""
    x = x.double()
    pairs = sum(sections)
    out, size = x.clone(), x.abs()
    for i in range(pairs):
        axis = next(a for a in range(len(sections)) if i < sum(sections[:a + 1]))
        angle = positions[axis].double() * inv_freq[i].double()
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        out[:, :, p] = x[:, :, p] * c - x[:, :, q] * s
        out[:, :, q] = x[:, :, q] * c + x[:, :, p] * s
        size[:, :, p] = size[:, :, q] = x[:, :, p].abs() + x[:, :, q].abs()
    return out, size


def attention_reference(q, k_pages, v_pages, k_scale, v_scale, sm_scale, offsets, lens, table,
                        num_pages):
    """In float64, one request and KV head at a time, for [T, Hq, D] queries:
      out, lse   the definition; positions of pages outside the pool are left out
      mean_abs   sum_s softmax_s |v_s|, what a relative error of p costs
      max_abs    the largest |v| seen, and
      terms      the largest sm_scale sum_d |q_d k_d| seen, of each row."""
    T, hq, d = q.shape
    hkv = k_pages.shape[1]
    g = hq // hkv
    f64 = dict(dtype=torch.float64, device=q.device)
    r = dict(out=torch.zeros(T, hq, d, **f64), lse=torch.full((T, hq), -float("inf"), **f64),
             mean_abs=torch.zeros(T, hq, d, **f64), max_abs=torch.zeros(T, hq, **f64),
             terms=torch.zeros(T, hq, **f64))
    for b in range(len(lens)):
        q0, n, length = offsets[b], offsets[b + 1] - offsets[b], lens[b]
        if n == 0 or length == 0:
            continue
        pages = table[b, :ceil_pages(length)].long()
        there = ((pages >= 0) & (pages < num_pages)).repeat_interleave(PAGE)[:length]
        if not bool(there.any()):
            continue
        pages = pages.clamp(0, num_pages - 1)
        pos = torch.arange(length, device=q.device)[there]
        last = torch.arange(length - n, length, device=q.device)
        hidden = (pos[None, :] > last[:, None])[:, None, :]
        for h in range(hkv):
            k = k_pages[pages, h].double().flatten(0, 1)[:length][there] * k_scale
            v = v_pages[pages, h].double().flatten(0, 1)[:length][there] * v_scale
            rows, heads = slice(q0, q0 + n), slice(h * g, (h + 1) * g)
            x = q[rows, heads].double() * sm_scale
            z = torch.einsum("tgd,sd->tgs", x, k).masked_fill(hidden, -float("inf"))
            sizes = torch.einsum("tgd,sd->tgs", x.abs(), k.abs()).masked_fill(hidden, 0.0)
            top = z.amax(-1, keepdim=True)
            seen = torch.isfinite(top)
            p = torch.where(seen, torch.exp(z - torch.where(seen, top, 0.0)), 0.0)
            total = p.sum(-1)
            p = p / total.clamp_min(1e-300)[..., None]
            r["out"][rows, heads] = torch.einsum("tgs,sd->tgd", p, v)
            r["mean_abs"][rows, heads] = torch.einsum("tgs,sd->tgd", p, v.abs())
            r["max_abs"][rows, heads] = torch.where(hidden, 0.0, v.abs().amax(-1)).amax(-1)
            r["terms"][rows, heads] = sizes.amax(-1)
            r["lse"][rows, heads] = torch.where(seen[..., 0], top[..., 0] + torch.log(total),
                                                -float("inf"))
    return r
