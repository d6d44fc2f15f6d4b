"""Plain references of the 8-bit cache with a scale for every 16 tokens of a head, written
from the definitions in include/dsa.h."""
import numpy as np
import torch

from paged_helpers import DEV, PAGE, ceil_pages

BLOCK = 16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
LARGEST = {E4M3: 448.0, INT8: 127.0}


def encode(x, code):
    """Codes nearest to fp32 values, saturating."""
    x = x.clamp(-LARGEST[code], LARGEST[code])
    return x.round().to(INT8) if code == INT8 else x.to(E4M3)


def decoded(codes, scales, which):
    """[pages, heads, 64, d] codes as float64 values; which: 0 keys, 1 values."""
    return codes.double() * scales[:, :, which].double().repeat_interleave(BLOCK, -1)[..., None]


def append_reference(pool, scales, which, slots, x):
    """The write of fp32 x [T, heads, d] into copies of a pool and its scales, token run by
    token run, in fp32 as the definition has it: (pool, scales, blocks written)."""
    pool, scales = pool.clone(), scales.clone()
    code = pool.dtype
    largest = torch.tensor(LARGEST[code])
    runs = {}
    for t, slot in enumerate(slots.tolist()):
        if slot >= 0:
            runs.setdefault(slot // BLOCK, []).append((t, slot % PAGE))
    for block, run in runs.items():
        page, part = divmod(block, PAGE // BLOCK)
        rows = [r for _, r in run]
        new = x[[t for t, _ in run]].cpu().transpose(0, 1)  # [heads, tokens, d]
        need = (new.abs().amax((1, 2)) / largest).clamp(2.0**-48, 2.0**32)
        scale = need
        if rows[0] % BLOCK:
            begun = scales[page, :, which, part].cpu()
            k = np.zeros(len(begun), dtype=np.int32)
            for h in range(len(begun)):
                while 2.0**-70 < float(begun[h]) * 2.0**k[h] < float(need[h]):
                    k[h] += 1
            k = torch.from_numpy(k)
            scale = begun * 2.0**k.float()
            old = slice(part * BLOCK, (part + 1) * BLOCK)
            held = pool.view(torch.uint8)[page, :, old].cpu().view(code).float()
            moved = encode(held * (2.0**-k.float())[:, None, None], code)
            pool.view(torch.uint8)[page, :, old] = moved.view(torch.uint8).to(DEV)
        scales[page, :, which, part] = scale.to(DEV)
        by = torch.ones(()) / scale
        codes = encode(new * by[:, None, None], code)
        pool.view(torch.uint8)[page, :, rows] = codes.view(torch.uint8).to(DEV)
    return pool, scales, list(runs)


def random_cache(g, pages, heads, d, code):
    """Codes near the end of their range, and scales that spread over a factor of ten."""
    x = torch.randn(2, pages, heads, PAGE, d, generator=g, device=DEV) * (LARGEST[code] / 3.75)
    codes = [encode(y, code) for y in x]
    spread = torch.randn(pages, heads, 2, PAGE // BLOCK, generator=g, device=DEV)
    return codes[0], codes[1], torch.exp(0.5 * spread) * 3.75 / LARGEST[code]


def slots_of(table, cached, new):
    """Slots of the new tokens of each request, in order."""
    out = []
    for b, (c, n) in enumerate(zip(cached, new)):
        out += [int(table[b, p // PAGE]) * PAGE + p % PAGE for p in range(c, c + n)]
    return torch.tensor(out, dtype=torch.int64, device=DEV)


def tables_of(g, lens, extra=2):
    """(table, number of pages) of requests of these lengths over shuffled pages."""
    counts = [ceil_pages(n) for n in lens]
    pages = sum(counts) + extra
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(counts))), -7, dtype=torch.int32, device=DEV)
    used = 0
    for b, c in enumerate(counts):
        table[b, :c] = ids[used:used + c]
        used += c
    return table, pages
