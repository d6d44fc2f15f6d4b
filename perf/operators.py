"""The paged key/value operators' cases: what is timed, on which inputs, and
what the results have to be.

Three operators of a dense-attention layer over 64-token pages, in the order a
serving step runs them:

  tables     request lengths -> block table, query offsets, cache slots, positions
  rope       rotary positions (1 to 3 axes) on q and k, k and v written into the pages
  attention  the new tokens' queries over every cached position, shared KV heads

`run` computes a case either from elementary torch operations in 32 bits (own is
False) or through the library's entry points (own is True).  `exact` is the
definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
PAGE = 64
MAX_SEQ = 1 << 20  # the longest context of the long-context workloads
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "fp8": 1}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one request's next token, in the middle of a page: pure call latency
        tables("tables one token", requests=1, cached=699, new=1, even=True, mix=1),
        # a full decode batch with five tokens to verify per request
        tables("tables 4096 verify", requests=4096, cached=16384, new=5, even=True, mix=2),
        # prompts entering together, 64 of them up to 32K tokens
        tables("tables 64 prompts", requests=64, cached=0, new=32768, even=False, mix=3),
        # one decode token of a 32/8-head layer
        rope("rope one token", tokens=1, hq=32, hkv=8, d=128, dtype="bf16", kv="bf16", rot=128,
             axes=1, start=131071),
        # an image-bearing prompt chunk: three axes, FP8 cache, a few padding rows
        rope("rope images", tokens=2048 + 5, hq=64, hkv=8, d=128, dtype="bf16", kv="fp8", rot=128,
             axes=3, start=777, pad=5),
        # a long prompt at the far end of the window, half the head rotated, pairs interleaved
        rope("rope long prompt", tokens=32768, hq=32, hkv=4, d=256, dtype="f16", kv="f16", rot=128,
             axes=1, start=MAX_SEQ - 32768, interleaved=True),
        # one short chat: latency
        attention("attn one short", requests=1, length=700, hq=32, hkv=8, d=128, dtype="bf16",
                  kv="bf16"),
        # one request over the whole 1M window
        attention("attn 1M", requests=1, length=MAX_SEQ, hq=32, hkv=8, d=128, dtype="bf16",
                  kv="bf16"),
        # a ragged decode batch over FP8 pages, two slots of it padding
        attention("attn ragged fp8", requests=64, length=32768, hq=64, hkv=8, d=128, dtype="bf16",
                  kv="fp8", even=False, mix=5, pad=2),
        # five tokens per request to verify, 131072-token agentic contexts
        attention("attn verify", requests=16, length=131072, new=5, hq=64, hkv=8, d=128,
                  dtype="bf16", kv="bf16", even=False, mix=6),
        # plain multi-head attention with narrow heads and odd lengths
        attention("attn heads64 f16", requests=37, length=4111, hq=16, hkv=16, d=64, dtype="f16",
                  kv="f16", even=False, mix=7),
        # one rank's 12 of 96 heads on one shared, wide KV head
        attention("attn shared head", requests=32, length=16384, hq=12, hkv=1, d=256,
                  dtype="bf16", kv="fp8", even=False, mix=8),
    ]


def tables(name, requests, cached, new, even, mix, pad=0):
    return dict(name=name, op="tables", requests=requests, cached=cached, new=new, even=even,
                mix=mix, pad=pad)


def rope(name, tokens, hq, hkv, d, dtype, kv, rot, axes, start, interleaved=False, pad=0):
    return dict(name=name, op="rope", tokens=tokens, hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv,
                rot=rot, axes=axes, start=start, interleaved=interleaved, pad=pad)


def attention(name, requests, length, hq, hkv, d, dtype, kv, new=1, even=True, mix=0, pad=0):
    return dict(name=name, op="attention", requests=requests, length=length, new=new, hq=hq,
                hkv=hkv, d=d, dtype=dtype, kv=kv, even=even, mix=mix, pad=pad)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "attention", "attention"])
    if op == "tables":
        requests = _log(rng, 1, 4096)
        new = _log(rng, 1, max(1, min(32768, (1 << 20) // requests)))
        cached = rng.choice([0, _log(rng, 1, 65536)])
        c = tables("", requests, cached, new, rng.random() < 0.3, rng.randrange(1 << 20),
                   rng.choice([0, 0, 3]))
    else:
        hkv = rng.choice([1, 2, 4, 5, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        d = rng.choice([64, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        kv = rng.choice([dtype, "fp8"])
        if op == "rope":
            axes = rng.choice([1, 1, 2, 3])
            rot = 16 * rng.randint(axes, d // 16)
            c = rope("", _log(rng, 1, 32768), hkv * group, hkv, d, dtype, kv, rot, axes,
                     _log(rng, 1, MAX_SEQ) - 1, rng.random() < 0.4, 0)
            c["pad"] = rng.choice([0, 0, min(3, c["tokens"] - 1)])
        else:
            new = rng.choice([1, 1, 1, 2, 3, 5, 8])
            requests = _log(rng, 1, 256)
            c = attention("", requests, _log(rng, max(8, new), 131072), hkv * group, hkv, d, dtype,
                          kv, new, rng.random() < 0.3, rng.randrange(1 << 20),
                          rng.choice([0, 0, 1, 3]))
    del c["name"]
    largest = {"tables": 0, "rope": 1, "attention": 2}[op]
    cap = [work(x) for x in listed() if x["op"] == op]
    cap = {k: max(w[k] for w in cap) for k in ("bytes", "flops")}
    size = ("new", "tokens", "length")[largest]
    while any(work(c)[k] > cap[k] for k in cap) or (op == "attention" and _plain_bytes(c) > 24e9):
        if c[size] > 16:
            c[size] //= 2
        elif op == "tables":
            c["requests"] //= 2
        else:
            c["hq"], c["hkv"] = 16, 1
    return c


def _plain_bytes(c):
    """The plain attention's largest intermediates."""
    pages = sum(-(-n // PAGE) for n in _lengths(c)[0])
    rows = c["new"] * c["hq"] // c["hkv"]
    return pages * c["hkv"] * 4 * (2 * PAGE * c["d"] + 3 * rows * PAGE + rows * c["d"])


def _spread(rng, top, even):
    """A length of 1..top: all of it, or mostly spread over the last factor of eight."""
    if even or top <= 1:
        return top
    return top if rng.random() < 0.1 else max(1, int(top * 2 ** rng.uniform(-3, 0)))


def _lengths(c):
    """Per request of an attention case: (context length, new tokens).  Padding
    requests have query rows and no context at all."""
    rng = random.Random(c["mix"])
    lens = [max(c["new"], _spread(rng, c["length"], c["even"])) for _ in range(c["requests"])]
    return lens + [0] * c["pad"], [c["new"]] * (c["requests"] + c["pad"])


def _growth(c):
    """Per request of a tables case: (cached tokens, new tokens).  Padding
    requests have neither."""
    rng = random.Random(c["mix"])
    cached = [_spread(rng, c["cached"], False) if c["cached"] else 0 for _ in range(c["requests"])]
    new = [_spread(rng, c["new"], c["even"]) for _ in range(c["requests"])]
    return cached + [0] * c["pad"], new + [0] * c["pad"]


def work(c):
    if c["op"] == "tables":
        cached, new = _growth(c)
        taken = sum(_pages(a + n) - _pages(a) for a, n in zip(cached, new))
        partial = sum(1 for a in cached if a % PAGE)
        # lengths, free pages and open pages read; table entries, offsets and lengths,
        # and per token a slot, a position and its request written
        return {"bytes": 16 * len(new) + 4 + 8 * taken + 4 * partial + 16 * sum(new),
                "flops": 0}
    e, s = SIZE[c["dtype"]], SIZE[c["kv"]]
    if c["op"] == "rope":
        t, stored = c["tokens"], c["tokens"] - c["pad"]
        values = t * c["hq"] + stored * c["hkv"]
        return {"bytes": t * 2 * c["hq"] * c["d"] * e + stored * 2 * c["hkv"] * c["d"] * (e + s) +
                t * (8 + 4 * c["axes"]) + 4 * c["rot"],
                "flops": 3 * values * c["rot"]}
    lens, new = _lengths(c)
    seen = sum(n * s_ - n * (n - 1) // 2 for s_, n in zip(lens, new) if s_)
    return {"bytes": 2 * sum(lens) * c["hkv"] * c["d"] * s + sum(new) * c["hq"] *
            (2 * c["d"] * e + 4) + 4 * sum(_pages(n) for n in lens),
            "flops": 4 * seen * c["hq"] * c["d"]}


def _pages(n):
    return -(-n // PAGE)


# ---- inputs -----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    state = {"tables": _prepare_tables, "rope": _prepare_rope,
             "attention": _prepare_attention}[case["op"]](case, g)
    state["case"] = case
    if own:
        _own_calls(state)
    return state


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _prepare_tables(c, g):
    cached, new = _growth(c)
    held = [_pages(a) for a in cached]
    grown = [_pages(a + n) - h for a, n, h in zip(cached, new, held)]
    total, width = sum(held) + sum(grown), max(h + k for h, k in zip(held, grown)) + 3
    pages = torch.randperm(total + 7, generator=g, device=DEV).to(torch.int32)
    have = torch.arange(width, device=DEV) < torch.tensor(held, device=DEV)[:, None]
    table = torch.full((len(new), width), -1, dtype=torch.int32, device=DEV)
    table[have] = pages[:sum(held)]
    tokens = sum(new)
    return dict(cached=_int32(cached), new=_int32(new), free=pages[sum(held):].contiguous(),
                num_pages=total + 7, tokens=tokens, grown=sum(grown), table=table,
                q_offsets=_int32([0] * (len(new) + 1)), seq_lens=_int32([0] * len(new)),
                slots=torch.zeros(tokens, dtype=torch.int64, device=DEV),
                positions=_int32([0]).repeat(tokens), requests=_int32([0]).repeat(tokens),
                taken=_int32([0]), status=_int32([0]))


def _normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _pool(g, pages, hkv, d, kv, scale):
    """A cache pool whose values (codes times scale) are standard normal."""
    x = _normal(g, pages, hkv, PAGE, d, dtype=torch.float16 if kv == "f16" else torch.bfloat16)
    return x if kv != "fp8" else (x / scale).to(torch.float8_e4m3fn)


def _prepare_rope(c, g):
    t, d, rot, axes = c["tokens"], c["d"], c["rot"], c["axes"]
    dt = DTYPE[c["dtype"]]
    pages = _pages(t + 37) + 1
    qkv = _normal(g, t, c["hq"] + 2 * c["hkv"], d, dtype=dt)  # one fused projection
    q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
    # tokens in order over shuffled pages, starting inside one; the last rows are padding
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(t, device=DEV) + 37
    slots = order[at // PAGE] * PAGE + at % PAGE
    slots[t - c["pad"]:] = -1
    i = torch.arange(t, device=DEV, dtype=torch.int32)
    if axes == 1:
        positions = (c["start"] + i)[None]
    else:  # frames of 24 x 36 patches (two axes: rows of 36)
        grid = [i // (24 * 36), i // 36 % 24, i % 36][3 - axes:] if axes == 3 else [i // 36, i % 36]
        positions = torch.stack([c["start"] + x for x in grid])
    pairs = rot // 2
    sections = [pairs // axes] * axes
    sections[-1] += pairs - sum(sections)
    kd, vd = (0.02, 0.03) if c["kv"] == "fp8" else (1.0, 1.0)
    return dict(q=q, k=k, v=v, slots=slots, positions=positions.to(torch.int32).contiguous(),
                inv_freq=10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs),
                sections=sections, k_scale=kd, v_scale=vd,
                k_pages=_pool(g, pages, c["hkv"], d, c["kv"], kd),
                v_pages=_pool(g, pages, c["hkv"], d, c["kv"], vd),
                q_out=torch.empty(t, c["hq"], d, dtype=dt, device=DEV), status=_int32([0]))


def _prepare_attention(c, g):
    lens, new = _lengths(c)
    counts = [_pages(n) for n in lens]
    pages, width = sum(counts) + 2, max(max(counts), 1)
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
    have = torch.arange(width, device=DEV) < torch.tensor(counts, device=DEV)[:, None]
    table[have] = ids[:sum(counts)]
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    kd, vd = (0.02, 0.03) if c["kv"] == "fp8" else (1.0, 1.0)
    dt = DTYPE[c["dtype"]]
    tokens = offsets[-1]
    # queries twice as long as the keys: scores spread over +-6, a few positions dominate
    return dict(q=2 * _normal(g, tokens, c["hq"], c["d"], dtype=dt),
                k_pages=_pool(g, pages, c["hkv"], c["d"], c["kv"], kd),
                v_pages=_pool(g, pages, c["hkv"], c["d"], c["kv"], vd),
                k_scale=kd, v_scale=vd, sm_scale=1 / math.sqrt(c["d"]),
                table=table, q_offsets=_int32(offsets), seq_lens=_int32(lens), lens=lens, new=new,
                num_pages=pages, num_table=sum(counts),
                out=torch.empty(tokens, c["hq"], c["d"], dtype=dt, device=DEV),
                lse=torch.empty(tokens, c["hq"], dtype=torch.float32, device=DEV),
                status=_int32([0]))


# ---- through the library ----------------------------------------------------

def _own_calls(s):
    """The prepared call a serving loop keeps for a step on the same buffers."""
    import dsa_sparse_attention_step_gb300 as dsa
    c = s["case"]
    if c["op"] == "tables":
        s["call"] = dsa.prepare_build_tables(
            s["cached"], s["new"], s["free"], s["num_pages"], s["table"], s["q_offsets"],
            s["seq_lens"], s["slots"], s["positions"], s["requests"], s["taken"], s["status"])
        return
    cache = dsa.KvCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if c["op"] == "rope":
        plan = dsa.Rope(s["inv_freq"], s["sections"], c["interleaved"])
        s["call"] = dsa.prepare_rope_append(cache, plan, s["positions"], s["slots"], s["q"],
                                            s["k"], s["v"], s["q_out"], s["status"])
        return
    batch = dsa.Batch(s["q_offsets"], s["seq_lens"], s["table"], s["num_pages"], s["lens"],
                      s["new"])
    need = dsa.dsa_paged_attention_workspace_size(batch, cache, c["hq"])
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    s["call"] = dsa.prepare_paged_attention(batch, cache, s["q"], s["sm_scale"], s["out"],
                                            s["lse"], ws, s["status"])


def run(state):
    op = state["case"]["op"]
    if own:
        state["call"]()
    else:
        {"tables": _plain_tables, "rope": _plain_rope, "attention": _plain_attention}[op](state)
    if op == "tables":
        return {k: state[k] for k in ("table", "q_offsets", "seq_lens", "slots", "positions",
                                      "requests", "taken")}
    if op == "rope":
        return {k: state[k] for k in ("q_out", "k_pages", "v_pages")}
    return {k: state[k] for k in ("out", "lse")}


# ---- plain forms ------------------------------------------------------------

def _plain_tables(s):
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    ends = new.cumsum(0)
    s["q_offsets"][1:] = ends
    s["seq_lens"].copy_(cached + new)
    held = (cached + PAGE - 1) // PAGE
    grown = (cached + new + PAGE - 1) // PAGE - held
    # the i-th new page goes to the request whose range of new pages holds i
    every = torch.arange(new.numel(), device=DEV)
    row = torch.repeat_interleave(every, grown, output_size=s["grown"])
    nth = torch.arange(s["grown"], device=DEV)
    col = held[row] + nth - (grown.cumsum(0) - grown)[row]
    table[row, col] = s["free"][nth]
    s["taken"].copy_(grown.sum())
    owner = torch.repeat_interleave(every, new, output_size=s["tokens"])
    pos = cached[owner] + torch.arange(s["tokens"], device=DEV) - (ends - new)[owner]
    s["slots"].copy_(table[owner, pos // PAGE].long() * PAGE + pos % PAGE)
    s["positions"].copy_(pos)
    s["requests"].copy_(owner)


def _turn(x, cos, sin, rot, interleaved):
    """The first `rot` values of every head turned, pair by pair."""
    x = x.float()
    head = x[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else head.chunk(2, dim=-1)
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((head, x[..., rot:]), dim=-1)


def _stored(x, kv, scale):
    """What a cache of this type holds of x."""
    if kv == "fp8":
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.to(DTYPE[kv])


def _plain_rope(s):
    c = s["case"]
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=DEV),
                                   torch.tensor(s["sections"]).to(DEV),
                                   output_size=c["rot"] // 2)
    # positions reach 2^20: the angle needs more than 32 bits
    angle = s["positions"].double().T[:, axis] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["q_out"].copy_(_turn(s["q"], cos, sin, c["rot"], c["interleaved"]))
    k = _stored(_turn(s["k"], cos, sin, c["rot"], c["interleaved"]), c["kv"], s["k_scale"])
    v = _stored(s["v"].float(), c["kv"], s["v_scale"])
    n = c["tokens"] - c["pad"]
    page, row = s["slots"][:n] // PAGE, s["slots"][:n] % PAGE
    for pool, x in ((s["k_pages"], k), (s["v_pages"], v)):
        if c["kv"] == "fp8":
            pool, x = pool.view(torch.uint8), x.view(torch.uint8)
        pool[page, :, row] = x[:n]


def _plain_attention(s):
    c = s["case"]
    n, hkv, d = c["new"], c["hkv"], c["d"]
    group, requests = c["hq"] // hkv, len(s["lens"])
    lens = s["seq_lens"].long()
    pages = (lens + PAGE - 1) // PAGE
    # one entry per page of every request: its request, its first position, its keys and values
    owner = torch.repeat_interleave(torch.arange(requests, device=DEV), pages,
                                    output_size=s["num_table"])
    nth = torch.arange(s["num_table"], device=DEV) - (pages.cumsum(0) - pages)[owner]
    page = s["table"][owner, nth].long()
    k = s["k_pages"].view(torch.uint8)[page].view(s["k_pages"].dtype).float() * s["k_scale"]
    # queries as [request, KV head, (token, head of the group), d]
    q = s["q"].float().view(requests, n, hkv, group, d).transpose(1, 2)
    q = q.reshape(requests, hkv, n * group, d) * s["sm_scale"]
    score = q[owner] @ k.transpose(-1, -2)
    del k
    pos = nth[:, None] * PAGE + torch.arange(PAGE, device=DEV)
    last = lens[:, None] - n + torch.arange(n, device=DEV).repeat_interleave(group)
    seen = pos[:, None, None, :] <= last[owner][:, None, :, None]
    score = torch.where(seen, score, -math.inf)
    top = torch.full((requests, hkv, n * group), -math.inf, device=DEV)
    top.index_reduce_(0, owner, score.amax(-1), "amax")
    shift = torch.where(top.isinf(), 0.0, top)
    p = torch.exp(score - shift[owner][..., None])
    del score
    v = s["v_pages"].view(torch.uint8)[page].view(s["v_pages"].dtype).float() * s["v_scale"]
    total = torch.zeros_like(top).index_add_(0, owner, p.sum(-1))
    acc = torch.zeros(requests, hkv, n * group, d, device=DEV).index_add_(0, owner, p @ v)
    out = torch.where(total[..., None] > 0, acc / total[..., None], 0.0)
    lse = shift + torch.log(total)

    def tokens(x):  # back to [token, head, ...]
        x = x.view(requests, hkv, n, group, -1).transpose(1, 2)
        return x.reshape(requests * n, hkv * group, -1)
    s["out"].copy_(tokens(out))
    s["lse"].copy_(tokens(lse)[..., 0])


# ---- definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables" or work(case)["flops"] > 4e12:
        return None  # whole numbers; or too long in 64 bits
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_attention(case, s)


def _exact_rope(c, s):
    """Each rotated pair as a complex number times e^(i angle)."""
    angle, first = [], 0
    for a, count in enumerate(s["sections"]):
        freq = s["inv_freq"][first:first + count]
        angle.append(s["positions"][a].double()[:, None] * freq)
        first += count
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=DEV).expand(c["tokens"], first),
                       torch.cat(angle, 1))[:, None]

    def turned(x):
        x = x.double().clone()
        if c["interleaved"]:
            a, b = slice(0, c["rot"], 2), slice(1, c["rot"], 2)
        else:
            a, b = slice(0, c["rot"] // 2), slice(c["rot"] // 2, c["rot"])
        z = torch.complex(x[..., a], x[..., b]) * unit
        x[..., a], x[..., b] = z.real, z.imag
        return x
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    at = [divmod(i, PAGE) for i in s["slots"].tolist()]
    keep = [i for i, (page, _) in enumerate(at) if page >= 0]
    page = torch.tensor([at[i][0] for i in keep], device=DEV)
    row = torch.tensor([at[i][1] for i in keep], device=DEV)
    for pool, x, scale in ((k_pages, turned(s["k"]), s["k_scale"]),
                           (v_pages, s["v"].double(), s["v_scale"])):
        x = x[keep]
        pool[page, :, row] = (x / scale).clamp(-448, 448) if c["kv"] == "fp8" else x
    return {"q_out": turned(s["q"]), "k_pages": k_pages, "v_pages": v_pages}


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
            k, v = (x[pages, h].double().flatten(0, 1)[:length] * f for x, f in
                    ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            heads = slice(h * group, (h + 1) * group)
            z = torch.einsum("tgd,sd->tgs", s["q"][rows, heads].double(), k) * s["sm_scale"]
            z.masked_fill_(later[:, None], -math.inf)
            lse[rows, heads] = torch.logsumexp(z, -1)
            out[rows, heads] = torch.einsum("tgs,sd->tgd", torch.softmax(z, -1), v)
    return {"out": out, "lse": lse}
