"""Cases of the 8-bit key/value cache whose scales follow the data: what is timed,
on which inputs, and what the results have to be.

A cache holds keys and values as E4M3 or INT8 codes in 64-token pages, with a scale
for every 16 tokens (a block) of a head.  Three operators use it:

  append     rotary positions on q and k, k and v quantised as they are written; a block
             that is fresh takes its scale from its tokens, one that was begun doubles
             its scale until they fit, and its older codes follow
  read       the values of a range of positions, as 16-bit rows
  attention  the new tokens' queries over every cached position, shared KV heads

Append cases of INT8 caches read back what they touched: codes of eight bits are
compared as the values they stand for.

`run` computes a case either from elementary torch operations in 32 bits (own is
False) or through the library's entry points (own is True).  `exact` is the
definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
PAGE, BLOCK = 64, 16
MAX_SEQ = 1 << 20  # the longest context of the long-context workloads
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LARGEST = {"e4m3": 448.0, "int8": 127.0}
SCALE_MIN, SCALE_MAX = 2.0 ** -48, 2.0 ** 32


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one request's next token, in the middle of a block: pure call latency
        append("append one token", requests=1, cached=699, new=1, hq=32, hkv=8, d=128,
               dtype="bf16", code="e4m3", rot=128),
        # a long prompt after a short cached prefix
        append("append prompt", requests=1, cached=37, new=32768, hq=32, hkv=8, d=128,
               dtype="bf16", code="e4m3", rot=128),
        # a decode batch with up to five tokens to verify per request, some rows padding
        append("append verify int8", requests=256, cached=16384, new=5, hq=64, hkv=8, d=128,
               dtype="bf16", code="int8", rot=128, mix=3, pad=3, read=True),
        # prompts of several requests, wide heads rotated by half in interleaved pairs
        append("append prompts int8", requests=7, cached=1000, new=4096, hq=16, hkv=4, d=256,
               dtype="f16", code="int8", rot=128, interleaved=True, mix=4, pad=2, read=True),
        # a short chat's keys and values, to hand to another program
        read("read short", requests=1, length=700, hkv=8, d=128, dtype="bf16", code="e4m3"),
        # long prefixes
        read("read long int8", requests=3, length=131072, hkv=8, d=128, dtype="bf16", code="int8",
             mix=5),
        # one short chat: latency
        attention("attn one short", requests=1, length=700, hq=32, hkv=8, d=128, dtype="bf16",
                  code="e4m3"),
        # one request over the whole 1M window
        attention("attn 1M int8", requests=1, length=MAX_SEQ, hq=32, hkv=8, d=128, dtype="bf16",
                  code="int8"),
        # a ragged decode batch, two slots of it padding
        attention("attn ragged", requests=64, length=32768, hq=64, hkv=8, d=128, dtype="bf16",
                  code="e4m3", mix=6, pad=2),
        # up to five tokens per request to verify, 131072-token agentic contexts
        attention("attn verify int8", requests=16, length=131072, new=5, hq=64, hkv=8, d=128,
                  dtype="bf16", code="int8", mix=7),
        # one rank's 12 of 96 heads on one shared, wide KV head
        attention("attn shared head int8", requests=32, length=16384, hq=12, hkv=1, d=256,
                  dtype="f16", code="int8", mix=8),
        # a prompt chunk over what is cached of its request
        attention("attn chunk", requests=1, length=16384, new=1000, hq=32, hkv=8, d=128,
                  dtype="bf16", code="e4m3", even=True),
    ]


def append(name, requests, cached, new, hq, hkv, d, dtype, code, rot, axes=1, interleaved=False,
           even=False, mix=0, pad=0, read=False):
    return dict(name=name, op="append", requests=requests, cached=cached, new=new, hq=hq, hkv=hkv,
                d=d, dtype=dtype, code=code, rot=rot, axes=axes, interleaved=interleaved,
                even=even or requests == 1, mix=mix, pad=pad, read=read)


def read(name, requests, length, hkv, d, dtype, code, even=False, mix=0):
    return dict(name=name, op="read", requests=requests, length=length, hkv=hkv, d=d, dtype=dtype,
                code=code, even=even or requests == 1, mix=mix)


def attention(name, requests, length, hq, hkv, d, dtype, code, new=1, even=False, mix=0, pad=0):
    return dict(name=name, op="attention", requests=requests, length=length, new=new, hq=hq,
                hkv=hkv, d=d, dtype=dtype, code=code, even=even or requests == 1, mix=mix, pad=pad)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attention", "attention", "attention"])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    d = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    code = rng.choice(["e4m3", "int8"])
    mix = rng.randrange(1 << 20)
    if op == "append":
        requests = _log(rng, 1, 512)
        axes = rng.choice([1, 1, 2, 3])
        c = append("", requests, _log(rng, 1, MAX_SEQ // 2) - 1,
                   _log(rng, 1, max(1, min(32768, 65536 // requests))), hkv * group, hkv, d, dtype,
                   code, rng.choice([0, 16 * rng.randint(axes, d // 16)]), axes,
                   rng.random() < 0.4, rng.random() < 0.3, mix, rng.choice([0, 0, 3]),
                   code == "int8")
    elif op == "read":
        c = read("", _log(rng, 1, 128), _log(rng, 1, 131072), hkv, d, dtype, code,
                 rng.random() < 0.3, mix)
    else:
        chunk = rng.random() < 0.25
        new = _log(rng, 16, 1000) if chunk else rng.choice([1, 1, 1, 2, 3, 5, 8])
        c = attention("", _log(rng, 1, 6 if chunk else 256),
                      _log(rng, max(8, new), 32768 if chunk else 131072), hkv * group, hkv, d,
                      dtype, code, new, rng.random() < 0.3, mix, rng.choice([0, 0, 1, 3]))
    del c["name"]
    cap = [work(x) for x in listed() if x["op"] == op]
    cap = {k: max(w[k] for w in cap) for k in ("bytes", "flops")}
    size = {"append": "new", "read": "length", "attention": "length"}[op]
    while any(work(c)[k] > cap[k] for k in cap) or (op == "attention" and _plain_bytes(c) > 24e9):
        if c[size] > 64:
            c[size] //= 2
        elif c["requests"] > 1:
            c["requests"] //= 2
        else:
            c["hkv"], c["hq"] = 1, 8
        if op == "attention":
            c["new"] = min(c["new"], c["length"])
    return c


def _plain_bytes(c):
    """The plain attention's largest intermediates."""
    pages = sum(_pages(n) for n in _lengths(c)[0])
    rows = c["new"] * c["hq"] // c["hkv"]
    return pages * c["hkv"] * 4 * (2 * PAGE * c["d"] + 3 * rows * PAGE + rows * c["d"])


def _spread(rng, top, even):
    """A length of 1..top: all of it, or mostly spread over the last factor of eight."""
    if even or top <= 1:
        return top
    return top if rng.random() < 0.1 else max(1, int(top * 2 ** rng.uniform(-3, 0)))


def _lengths(c):
    """Per request of a read or attention case: (context length, new tokens).  Padding
    requests have query rows and no context at all."""
    rng = random.Random(c["mix"])
    new = [c.get("new", 1) if c["even"] else rng.randint(1, c.get("new", 1))
           for _ in range(c["requests"])]
    lens = [max(n, _spread(rng, c["length"], c["even"])) for n in new]
    pad = c.get("pad", 0)
    return lens + [0] * pad, new + [1] * pad


def _growth(c):
    """Per request of an append case: (cached tokens, new tokens)."""
    rng = random.Random(c["mix"])
    cached = [_spread(rng, c["cached"], c["even"]) if c["cached"] else 0
              for _ in range(c["requests"])]
    return cached, [_spread(rng, c["new"], c["even"]) for _ in range(c["requests"])]


def _pages(n):
    return -(-n // PAGE)


def work(c):
    e = 2
    if c["op"] == "append":
        cached, new = _growth(c)
        t = sum(new) + c["pad"]
        blocks = sum((a + n - 1) // BLOCK - a // BLOCK + 1 for a, n in zip(cached, new))
        b = (t * (2 * c["hq"] * c["d"] * e + 8 + 4 * c["axes"] * (c["rot"] > 0)) + 4 * c["rot"] +
             sum(new) * 2 * c["hkv"] * c["d"] * (e + 1) + blocks * c["hkv"] * 8)
        if c["read"]:  # and what stands before the new tokens in their blocks, written out too
            old = sum(a % BLOCK for a in cached)
            b += 2 * c["hkv"] * c["d"] * ((sum(new) + old) * e + old)
        values = t * c["hq"] + sum(new) * c["hkv"]
        return {"bytes": b, "flops": 3 * values * c["rot"]}
    lens, new = _lengths(c)
    held = 2 * sum(lens) * c["hkv"] * c["d"]
    scales = 8 * c["hkv"] * sum(-(-n // BLOCK) for n in lens)
    table = 4 * sum(_pages(n) for n in lens)
    if c["op"] == "read":
        return {"bytes": held * (1 + e) + scales + table, "flops": held}
    seen = sum(n * s - n * (n - 1) // 2 for s, n in zip(lens, new) if s)
    return {"bytes": held + scales + table + sum(new) * c["hq"] * (2 * c["d"] * e + 4),
            "flops": 4 * seen * c["hq"] * c["d"]}


# ---- inputs -----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    state = (_prepare_append if case["op"] == "append" else _prepare_context)(case, g)
    state["case"] = case
    if own:
        _own_calls(state)
    return state


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _pool(c, pages, g):
    """Codes of a cache's keys or values: a block's largest is near the end of the range."""
    x = _normal(g, pages, c["hkv"], PAGE, c["d"], dtype=torch.bfloat16)
    x *= LARGEST[c["code"]] / 3.75
    x.clamp_(-LARGEST[c["code"]], LARGEST[c["code"]])
    return (x.round_() if c["code"] == "int8" else x).to(CODE[c["code"]])


def _scales(c, pages, g):
    """[page, head, keys or values, block]: values of about unit size, some blocks larger."""
    return torch.exp(0.4 * _normal(g, pages, c["hkv"], 2, PAGE // BLOCK)) * (
        3.75 / LARGEST[c["code"]])


def _offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _prepare_append(c, g):
    cached, new = _growth(c)
    tokens, d, dt, code = sum(new), c["d"], DTYPE[c["dtype"]], c["code"]
    # the pages that the new tokens touch, shuffled; the others of a context play no part
    first = [a // PAGE for a in cached]
    taken = [_pages(a + n) - f for a, n, f in zip(cached, new, first)]
    pages = sum(taken) + 1
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    begin = _offsets(taken)
    # per token: request, position, page entry, slot
    owner = torch.repeat_interleave(torch.arange(len(new), device=DEV),
                                    torch.tensor(new, device=DEV))
    pos = torch.arange(tokens, device=DEV) - torch.tensor(_offsets(new)[:-1], device=DEV)[owner]
    pos = pos + torch.tensor(cached, device=DEV)[owner]
    entry = pos // PAGE - torch.tensor(first, device=DEV)[owner] + torch.tensor(
        begin[:-1], device=DEV)[owner]
    slots = ids[entry].long() * PAGE + pos % PAGE
    # touched blocks in the order of the tokens, and every token's place among them
    block = slots // BLOCK
    starts = torch.ones(tokens, dtype=torch.bool, device=DEV)
    starts[1:] = block[1:] != block[:-1]
    # the last rows are padding
    rows = tokens + c["pad"]
    at = torch.cat((pos, pos.new_zeros(c["pad"])))
    slots = torch.cat((slots, slots.new_full((c["pad"],), -1)))
    if c["axes"] == 1:
        positions = at[None]
    else:  # frames of 24 x 36 patches (two axes: rows of 36)
        grid = [at // (24 * 36), at // 36 % 24, at % 36]
        positions = torch.stack(grid if c["axes"] == 3 else [at // 36, at % 36])
    pairs = c["rot"] // 2
    sections = [pairs // c["axes"]] * c["axes"]
    sections[-1] += pairs - sum(sections)
    qkv = _normal(g, rows, c["hq"] + 2 * c["hkv"], d, dtype=dt)  # one fused projection
    q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
    k *= torch.exp(0.5 * _normal(g, c["hkv"], d)).to(dt)  # keys have channels that stand out
    s = dict(q=q, k=k, v=v, slots=slots, positions=positions.to(torch.int32).contiguous(),
             inv_freq=10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) /
                                  max(pairs, 1)),
             sections=sections, blocks=block[starts], nth=starts.long().cumsum(0) - 1,
             tokens=tokens, k_pages=_pool(c, pages, g), v_pages=_pool(c, pages, g),
             scales=_scales(c, pages, g),
             q_out=torch.empty(rows, c["hq"], d, dtype=dt, device=DEV), status=_int32([0]))
    if c["read"]:  # from the beginning of the first touched block on
        lens = [a + n for a, n in zip(cached, new)]
        counts = [n + a % BLOCK for a, n in zip(cached, new)]
        width = max(_pages(n) for n in lens)
        table = torch.zeros(len(new), width, dtype=torch.int32, device=DEV)
        col = torch.arange(width, device=DEV) - torch.tensor(first, device=DEV)[:, None]
        have = (col >= 0) & (col < torch.tensor(taken, device=DEV)[:, None])
        table[have] = ids[:sum(taken)]
        s.update(_rows_out(c, table, lens, counts, pages))
    return s


def _rows_out(c, table, lens, counts, pages):
    """What reading each request's last `counts` positions takes."""
    shape = (sum(counts), c["hkv"], c["d"])
    return dict(table=table, offsets=_int32(_offsets(counts)), seq_lens=_int32(lens), lens=lens,
                new=counts, num_pages=pages,
                k_out=torch.empty(shape, dtype=DTYPE[c["dtype"]], device=DEV),
                v_out=torch.empty(shape, dtype=DTYPE[c["dtype"]], device=DEV))


def _prepare_context(c, g):
    lens, new = _lengths(c)
    counts = [_pages(n) for n in lens]
    pages, width = sum(counts) + 2, max(max(counts), 1)
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
    have = torch.arange(width, device=DEV) < torch.tensor(counts, device=DEV)[:, None]
    table[have] = ids[:sum(counts)]
    s = dict(k_pages=_pool(c, pages, g), v_pages=_pool(c, pages, g), scales=_scales(c, pages, g),
             status=_int32([0]))
    if c["op"] == "read":
        s.update(_rows_out(c, table, lens, lens, pages))
        return s
    tokens, dt = sum(new), DTYPE[c["dtype"]]
    # queries twice as long as the keys: scores spread over +-6, a few positions dominate
    s.update(q=2 * _normal(g, tokens, c["hq"], c["d"], dtype=dt), sm_scale=1 / math.sqrt(c["d"]),
             table=table, offsets=_int32(_offsets(new)), seq_lens=_int32(lens), lens=lens, new=new,
             num_pages=pages, num_table=sum(counts),
             out=torch.empty(tokens, c["hq"], c["d"], dtype=dt, device=DEV),
             lse=torch.empty(tokens, c["hq"], dtype=torch.float32, device=DEV))
    return s


# ---- through the library ----------------------------------------------------

def _own_calls(s):
    """The prepared calls that a serving loop keeps for a step on the same buffers."""
    import dsa_sparse_attention_step_gb300 as dsa
    c = s["case"]
    cache = dsa.QuantCache(s["k_pages"], s["v_pages"], s["scales"])
    s["calls"] = []
    if c["op"] == "append":
        rope = dsa.Rope(s["inv_freq"], s["sections"], c["interleaved"]) if c["rot"] else None
        s["calls"].append(dsa.prepare_quant_append(
            cache, rope, s["positions"], s["slots"], s["q"], s["k"], s["v"], s["q_out"],
            s["status"]))
        if not c["read"]:
            return
    batch = dsa.Batch(s["offsets"], s["seq_lens"], s["table"], s["num_pages"], s["lens"], s["new"])
    if c["op"] != "attention":
        s["calls"].append(dsa.prepare_quant_read(batch, cache, s["k_out"], s["v_out"],
                                                 s["status"]))
        return
    need = dsa.dsa_quant_attention_workspace_size(batch, cache, c["hq"])
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    s["calls"].append(dsa.prepare_quant_attention(batch, cache, s["q"], s["sm_scale"], s["out"],
                                                  s["lse"], ws, s["status"]))


def run(state):
    c = state["case"]
    if own:
        for call in state["calls"]:
            call()
    elif c["op"] == "attention":
        _plain_attention(state)
    else:
        if c["op"] == "append":
            _plain_append(state)
        if c["op"] == "read" or c["read"]:
            _plain_read(state)
    if c["op"] == "attention":
        return {k: state[k] for k in ("out", "lse")}
    if c["op"] == "read":
        return {k: state[k] for k in ("k_out", "v_out")}
    names = ("k_out", "v_out") if c["read"] else ("k_pages", "v_pages")
    return {k: state[k] for k in ("q_out", "scales") + names}


# ---- plain forms ------------------------------------------------------------

def _turn(x, cos, sin, rot, interleaved):
    """The first `rot` values of every head turned, pair by pair."""
    x = x.float()
    head = x[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else head.chunk(2, dim=-1)
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((head, x[..., rot:]), dim=-1)


def _encode(x, code):
    x = x.clamp(-LARGEST[code], LARGEST[code])
    return x.round().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _bytes(x):
    return x.view(torch.uint8)


def _plain_append(s):
    c, n = s["case"], s["tokens"]
    k, q = s["k"].float(), s["q"]
    if c["rot"]:
        axis = torch.repeat_interleave(torch.arange(c["axes"], device=DEV),
                                       torch.tensor(s["sections"]).to(DEV),
                                       output_size=c["rot"] // 2)
        # positions reach 2^20: the angle needs more than 32 bits
        angle = s["positions"].double().T[:, axis] * s["inv_freq"]
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        q = _turn(q, cos, sin, c["rot"], c["interleaved"])
        k = _turn(k, cos, sin, c["rot"], c["interleaved"])
    s["q_out"].copy_(q)
    page, part = s["blocks"] // (PAGE // BLOCK), s["blocks"] % (PAGE // BLOCK)
    row = s["slots"][:n] % BLOCK
    nth, count = s["nth"], s["blocks"].numel()
    fresh = torch.zeros(count, dtype=torch.int32, device=DEV).index_reduce_(
        0, nth, (row == 0).int(), "amax")[:, None] > 0
    for which, pool, x in ((0, s["k_pages"], k), (1, s["v_pages"], s["v"].float())):
        x = x[:n]
        top = torch.zeros(count, c["hkv"], device=DEV).index_reduce_(0, nth, x.abs().amax(-1),
                                                                     "amax")
        # (by a tensor: division by a number may be done as a product with its reciprocal)
        need = (top / torch.full_like(top, LARGEST[c["code"]])).clamp(SCALE_MIN, SCALE_MAX)
        old = s["scales"][page, :, which, part]
        (m0, e0), (m1, e1) = torch.frexp(old), torch.frexp(need)
        double = torch.where(fresh, 0, (e1 - e0 + (m1 > m0)).clamp_min(0))
        scale = torch.where(fresh, need, torch.ldexp(old, double))
        s["scales"][page, :, which, part] = scale
        blocks = pool.view(-1, c["hkv"], PAGE // BLOCK, BLOCK, c["d"])
        codes = blocks if c["code"] == "int8" else _bytes(blocks)
        held = codes[page, :, part].view(pool.dtype).float()
        held = torch.ldexp(held, -double[..., None, None])
        codes[page, :, part] = _encode(held, c["code"]).view(codes.dtype)
        new = _encode(x * (1 / scale)[nth][..., None], c["code"])
        codes[page[nth], :, part[nth], row] = new.view(codes.dtype)


def _plain_read(s):
    c = s["case"]
    lens, new = s["seq_lens"].long(), s["offsets"].long().diff()
    rows = s["k_out"].shape[0]
    owner = torch.repeat_interleave(torch.arange(lens.numel(), device=DEV), new, output_size=rows)
    pos = torch.arange(rows, device=DEV) - (s["offsets"][1:].long() - lens)[owner]
    page, row = s["table"][owner, pos // PAGE].long(), pos % PAGE
    for which, pool, out in ((0, s["k_pages"], s["k_out"]), (1, s["v_pages"], s["v_out"])):
        x = _bytes(pool)[page, :, row].view(pool.dtype).float()
        out.copy_(x * s["scales"][page, :, which, row // BLOCK][..., None])


def _plain_attention(s):
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    group, requests, n = c["hq"] // hkv, len(s["lens"]), max(s["new"])
    lens, new = s["seq_lens"].long(), s["offsets"].long().diff()
    pages = (lens + PAGE - 1) // PAGE
    # one entry per page of every request: its request, its first position, its keys and values
    owner = torch.repeat_interleave(torch.arange(requests, device=DEV), pages,
                                    output_size=s["num_table"])
    nth = torch.arange(s["num_table"], device=DEV) - (pages.cumsum(0) - pages)[owner]
    page = s["table"][owner, nth].long()

    def held(pool, which):
        scale = s["scales"][page, :, which].repeat_interleave(BLOCK, dim=-1)[..., None]
        return _bytes(pool)[page].view(pool.dtype).float() * scale
    # every request's queries, as many as the longest has, [request, KV head, (token, head), d]
    j = torch.arange(n, device=DEV)
    there = j < new[:, None]
    token = torch.where(there, s["offsets"][:-1].long()[:, None] + j, 0)
    q = s["q"].float()[token].view(requests, n, hkv, group, d).transpose(1, 2)
    q = q.reshape(requests, hkv, n * group, d) * s["sm_scale"]
    score = q[owner] @ held(s["k_pages"], 0).transpose(-1, -2)
    pos = nth[:, None] * PAGE + torch.arange(PAGE, device=DEV)
    last = torch.where(there, (lens - new)[:, None] + j, -1).repeat_interleave(group, dim=1)
    seen = pos[:, None, None, :] <= last[owner][:, None, :, None]
    score = torch.where(seen, score, -math.inf)
    top = torch.full((requests, hkv, n * group), -math.inf, device=DEV)
    top.index_reduce_(0, owner, score.amax(-1), "amax")
    shift = torch.where(top.isinf(), 0.0, top)
    p = torch.exp(score - shift[owner][..., None])
    del score
    total = torch.zeros_like(top).index_add_(0, owner, p.sum(-1))
    acc = torch.zeros(requests, hkv, n * group, d, device=DEV)
    acc.index_add_(0, owner, p @ held(s["v_pages"], 1))
    out = torch.where(total[..., None] > 0, acc / total[..., None], 0.0)
    lse = shift + torch.log(total)

    # back to [token, head, ...], without the rows that no token has
    rows = torch.arange(s["q"].shape[0], device=DEV)
    at = torch.repeat_interleave(torch.arange(requests, device=DEV), new,
                                 output_size=rows.numel())
    place = rows - s["offsets"][:-1].long()[at]

    def tokens(x):
        x = x.view(requests, hkv, n, group, -1).transpose(1, 2)
        return x[at, place].reshape(rows.numel(), hkv * group, -1)
    s["out"].copy_(tokens(out))
    s["lse"].copy_(tokens(lse)[..., 0])


# ---- definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None  # too long in 64 bits
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "read":
        return dict(zip(("k_out", "v_out"), _exact_read(case, s, _values(case, s))))
    return _exact_append(case, s)


def _values(c, s):
    """The whole cache's keys and values."""
    return [x.double() * s["scales"][:, :, i].double().repeat_interleave(BLOCK, -1)[..., None]
            for i, x in enumerate((s["k_pages"], s["v_pages"]))]


def _exact_read(c, s, values):
    """Request by request, its positions page by page."""
    out = [[], []]
    for b, (length, n) in enumerate(zip(s["lens"], s["new"])):
        pages = s["table"][b, :_pages(length)].long()
        for which, x in enumerate(values):
            first = (length - n) // PAGE  # pages before hold nothing that is read
            part = x[pages[first:]].transpose(1, 2).flatten(0, 1)
            out[which].append(part[length - n - first * PAGE:length - first * PAGE])
    return [torch.cat(x) for x in out]


def _exact_append(c, s):
    """Each rotated pair as a complex number times e^(i angle); then block by block."""
    pairs = c["rot"] // 2
    freq = s["inv_freq"].split(s["sections"])
    angle = torch.cat([s["positions"][a].double()[:, None] * f for a, f in enumerate(freq)], 1)
    unit = torch.complex(angle.cos(), angle.sin())[:, None]

    def turned(x):
        x = x.double().clone()
        a, b = ((slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if c["interleaved"]
                else (slice(0, pairs), slice(pairs, 2 * pairs)))
        z = torch.complex(x[..., a], x[..., b]) * unit
        x[..., a], x[..., b] = z.real, z.imag
        return x
    largest = LARGEST[c["code"]]

    def rounded(x):
        """To the nearest code, ties to the even one."""
        x = x.clamp(-largest, largest)
        if c["code"] == "int8":
            return x.round()
        step = torch.exp2(torch.log2(x.abs().clamp_min(2.0 ** -6)).floor() - 3)
        return (x / step).round() * step
    codes = [s["k_pages"].double(), s["v_pages"].double()]
    scales = s["scales"].double()
    new = [turned(s["k"]), s["v"].double()]
    runs = {}  # block -> its tokens
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            runs.setdefault(slot // BLOCK, []).append((t, slot % PAGE))
    for block, run_ in runs.items():
        page, part = divmod(block, PAGE // BLOCK)
        t = [i for i, _ in run_]
        row = torch.tensor([r for _, r in run_], device=DEV)
        old = slice(part * BLOCK, (part + 1) * BLOCK)
        for which in (0, 1):
            x = new[which][t[0]:t[-1] + 1].transpose(0, 1)  # [head, token, d]
            scale = (x.abs().amax((1, 2)) / largest).clamp(SCALE_MIN, SCALE_MAX)
            if run_[0][1] % BLOCK:
                begun = scales[page, :, which, part]
                times = torch.exp2(torch.log2(scale / begun).ceil().clamp_min(0))
                scale = begun * times
                codes[which][page, :, old] = rounded(codes[which][page, :, old] /
                                                     times[:, None, None])
            scales[page, :, which, part] = scale
            codes[which][page, :, row] = rounded(x / scale[:, None, None])
    out = {"q_out": turned(s["q"]), "scales": scales}
    if not c["read"]:
        return {**out, "k_pages": codes[0], "v_pages": codes[1]}
    values = [x * scales[:, :, i].repeat_interleave(BLOCK, -1)[..., None]
              for i, x in enumerate(codes)]
    return {**out, **dict(zip(("k_out", "v_out"), _exact_read(c, s, values)))}


def _exact_attention(c, s):
    """Request by request and head by head, softmax over the visible positions."""
    group = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for b, (length, n) in enumerate(zip(s["lens"], s["new"])):
        rows, first = slice(first, first + n), first + n
        if not length:
            continue
        pages = s["table"][b, :_pages(length)].long()
        later = torch.arange(length, device=DEV) > torch.arange(length - n, length,
                                                                device=DEV)[:, None]
        for h in range(c["hkv"]):
            k, v = (x[pages, h].double() * s["scales"][pages, h, i].double()
                    .repeat_interleave(BLOCK, -1)[..., None] for i, x in
                    enumerate((s["k_pages"], s["v_pages"])))
            k, v = k.flatten(0, 1)[:length], v.flatten(0, 1)[:length]
            for head in range(h * group, (h + 1) * group):
                z = (s["q"][rows, head].double() @ k.T) * s["sm_scale"]
                z.masked_fill_(later, -math.inf)
                lse[rows, head] = torch.logsumexp(z, -1)
                out[rows, head] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}
