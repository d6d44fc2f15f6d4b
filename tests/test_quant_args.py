"""Argument checks of the 8-bit cache's entry points (CPU only: every call here is refused
before anything is launched)."""
import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = ctypes.c_void_p(4096)  # never dereferenced
ODD = ctypes.c_void_p(4100)   # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    from dsa_sparse_attention_step_gb300 import _build
    _build.build()
    import dsa_sparse_attention_step_gb300 as dsa
    return dsa.load()


def _cache(**kw):
    import dsa_sparse_attention_step_gb300 as dsa
    c = dsa._CQuantCache(8, 2, 128, 0, 1 << 20, 2 << 20, 3 << 20)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _batch(**kw):
    import dsa_sparse_attention_step_gb300 as dsa
    b = dsa._CBatch(1, 1, 1, 4096, 8, 64, 64, 16, 32, 48)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _append(lib, cache=None, fmt=0, tokens=3, axes=1, sections=(64, 0, 0), freq=4096,
            positions=FAKE, slots=FAKE, hq=4, q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256,
            out=FAKE, os=512, rope=True):
    import dsa_sparse_attention_step_gb300 as dsa
    r = dsa._CRope(axes, (ctypes.c_int32 * 3)(*sections), 0, freq)
    c = _cache() if cache is None else cache
    return lib.dsa_quant_append(tokens, ctypes.byref(c), fmt, ctypes.byref(r) if rope else None,
                                positions, slots, hq, q, qs, k, ks, v, vs, out, os, None, None)


def _read(lib, cache=None, batch=None, fmt=0, k=FAKE, ks=256, v=FAKE, vs=256):
    c = _cache() if cache is None else cache
    return lib.dsa_quant_read(ctypes.byref(_batch(**(batch or {}))), ctypes.byref(c), fmt, k, ks,
                              v, vs, None, None)


def _attention(lib, cache=None, batch=None, fmt=0, hq=4, q=FAKE, qs=512, sm=0.1, out=FAKE,
               ws=FAKE, ws_bytes=1 << 40):
    c = _cache() if cache is None else cache
    return lib.dsa_quant_attention(ctypes.byref(_batch(**(batch or {}))), ctypes.byref(c), fmt, hq,
                                   q, qs, sm, out, None, ws, ws_bytes, None, None)


CACHE_REFUSALS = [
    (dict(head_dim=96), UNSUPPORTED), (dict(format=2), UNSUPPORTED), (dict(format=-1), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_pages=1 << 20, num_kv_heads=1 << 11), INVALID), (dict(k_pages=0), INVALID),
    (dict(k_pages=8200), INVALID), (dict(v_pages=8200), INVALID), (dict(scales=0), INVALID),
    (dict(scales=8196), INVALID)]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_cache_refusals(lib, kw, code):
    for call in (_append, _read, _attention):
        assert call(lib, cache=_cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(axes=4), UNSUPPORTED),
    (dict(axes=-1), UNSUPPORTED), (dict(sections=(-8, 0, 0)), INVALID),
    (dict(sections=(72, 0, 0)), INVALID), (dict(sections=(12, 0, 0)), UNSUPPORTED),
    (dict(rope=False), INVALID), (dict(freq=0), INVALID), (dict(positions=None), INVALID),
    (dict(slots=None), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID),
    (dict(qs=516), INVALID), (dict(qs=504), INVALID), (dict(ks=248), INVALID),
    (dict(vs=260), INVALID), (dict(k=ODD), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(os=500), INVALID), (dict(hq=-1), INVALID),
    (dict(hq=1 << 15, qs=1 << 22, os=1 << 22), UNSUPPORTED)])
def test_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=3), UNSUPPORTED), (dict(batch=dict(page_size=16)), UNSUPPORTED),
    (dict(batch=dict(num_pages=9)), INVALID), (dict(batch=dict(max_pages=3)), INVALID),
    (dict(k=ODD), INVALID), (dict(v=ODD), INVALID), (dict(ks=250), INVALID),
    (dict(vs=248), INVALID)])
def test_read_refusals(lib, kw, code):
    assert _read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=dict(page_size=32)), UNSUPPORTED), (dict(batch=dict(max_pages=10)), INVALID),
    (dict(batch=dict(num_pages=9)), INVALID), (dict(fmt=2), UNSUPPORTED), (dict(hq=0), INVALID),
    (dict(hq=5), INVALID), (dict(hq=1 << 15, qs=1 << 22), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(q=ODD), INVALID), (dict(qs=500), INVALID), (dict(sm=0.0), INVALID),
    (dict(sm=float("nan")), INVALID), (dict(sm=float("inf")), INVALID), (dict(sm=1e-39), INVALID),
    (dict(sm=3e38), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=ODD), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
    # 2^20 new tokens of one request, each over up to 2^20 positions
    (dict(batch=dict(total_q=1 << 20, max_q_per_request=1 << 20, max_seq_len=1 << 20,
                     max_pages=1 << 14)), UNSUPPORTED)])
def test_attention_refusals(lib, kw, code):
    assert _attention(lib, **kw) == code


@pytest.mark.parametrize("at,inside", [
    ((1 << 20), True), ((1 << 20) + 8 * 2 * 64 * 128 - 16, True), ((1 << 20) + 8 * 2 * 64 * 128, False),
    ((1 << 20) - 512, False), ((1 << 20) - 496, True), ((2 << 20) + 64, True),
    ((3 << 20) + 8 * 2 * 8 * 4 - 16, True), ((3 << 20) + 8 * 2 * 8 * 4, False)])
def test_outputs_inside_the_cache_are_refused(lib, at, inside):
    """(Those outside are let through these checks, and refused for a batch of another pool
    or for a missing key pointer.)"""
    p = ctypes.c_void_p(at)
    if inside:
        assert _read(lib, k=p) == INVALID and _read(lib, v=p) == INVALID
        assert _append(lib, tokens=1, hq=2, out=p, os=256) == INVALID
    else:
        assert _read(lib, k=p, batch=dict(total_q=0)) == 0


def test_calls_without_tokens_are_no_ops(lib):
    assert _append(lib, tokens=0) == 0
    assert _read(lib, batch=dict(total_q=0), k=None) == 0
    assert _read(lib, k=None, v=None) == 0
    assert _attention(lib, batch=dict(total_q=0), q=None, out=None, ws=None) == 0


def test_attention_workspace_follows_rows_and_head_dim(lib):
    b = _batch(num_requests=4, total_q=4)

    def size(hq, **kw):
        return lib.dsa_quant_attention_workspace_size(ctypes.byref(b), ctypes.byref(_cache(**kw)),
                                                      hq)
    assert 0 < size(4) <= size(64) <= size(128)
    assert size(4, head_dim=256) > size(4) > size(4, head_dim=64)
    assert size(5) == 0 and size(0) == 0 and size(4, head_dim=96) == 0


POOL = 8 * 2 * 64 * 128  # bytes of the keys' and of the values' codes of _cache()
K, V, S = 1 << 20, 2 << 20, 3 << 20


@pytest.mark.parametrize("begin,size", [(K, POOL), (V, POOL), (S, 8 * 2 * 8 * 4)])
@pytest.mark.parametrize("which", ["out", "lse", "ws"])
def test_attention_outputs_inside_the_cache_are_refused(lib, which, begin, size):
    """At its first and last bytes, in the middle and around it; apart from the address the
    call is one that the library takes."""
    b, c = _batch(), _cache()
    need = lib.dsa_quant_attention_workspace_size(ctypes.byref(b), ctypes.byref(c), 4)
    bytes_ = {"out": 4 * 128 * 2, "lse": 4 * 4, "ws": need}[which]
    step = 4 if which == "lse" else 16
    for at in (begin, begin + size - step, begin + size // 2, begin - bytes_ + step):
        if at <= 0:
            continue
        p = dict(out=1 << 40, lse=1 << 41, ws=1 << 42)
        p[which] = at // step * step
        assert lib.dsa_quant_attention(ctypes.byref(b), ctypes.byref(c), 0, 4, 1 << 43, 512, 0.1,
                                       p["out"], p["lse"], p["ws"], need, None, None) == INVALID


@pytest.mark.parametrize("a,b", [("out", "q"), ("lse", "q"), ("ws", "q"), ("out", "lse"), ("ws", "out"),
                                 ("ws", "lse"), ("out", "table"), ("lse", "lens"), ("ws", "offsets")])
def test_attention_outputs_that_overlap_are_refused(lib, a, b):
    batch, c = _batch(num_requests=3, total_q=3), _cache()
    need = lib.dsa_quant_attention_workspace_size(ctypes.byref(batch), ctypes.byref(c), 4)
    p = {name: (i + 1) << 40 for i, name in enumerate(("out", "lse", "ws", "q", "table", "lens",
                                                       "offsets"))}
    last = dict(q=3 * 2 * 512 - 16, lse=32, out=3 * 1024 - 16, table=3 * 64 * 4 - 16, lens=8, offsets=0)
    size = dict(out=3 * 1024, lse=48, ws=need)
    for at in (p[b], p[b] + last[b], p[b] - size[a] + 16):
        x = dict(p)
        x[a] = at // (4 if a == "lse" else 16) * (4 if a == "lse" else 16)
        batch.block_table, batch.seq_lens, batch.q_offsets = x["table"], x["lens"], x["offsets"]
        assert lib.dsa_quant_attention(ctypes.byref(batch), ctypes.byref(c), 0, 4, x["q"], 1024, 0.1,
                                       x["out"], x["lse"], x["ws"], need, None, None) == INVALID


FAR = [ctypes.c_void_p((i + 1) << 40) for i in range(6)]  # apart from one another and the cache


@pytest.mark.parametrize("at,qs,os", [
    (0, 512, 520), (16, 512, 512), (-1008, 512, 512), (2 * 520 * 2, 520, 520), (512, 1024, 2048),
    (2048 - 1008, 1024, 1024), (4096 - 2 * 1032 * 2, 1024, 1032)])
def test_queries_written_over_others_are_refused(lib, at, qs, os):
    """q_out begins `at` bytes behind q: three rows of 1024 bytes each, every so many values;
    over the first of q's rows, the last, or one in the middle."""
    assert _append(lib, tokens=3, hq=4, q=FAR[0], qs=qs, k=FAR[1], v=FAR[2], slots=FAR[3],
                   positions=FAR[4], freq=FAR[5].value, out=ctypes.c_void_p(FAR[0].value + at),
                   os=os) == INVALID


@pytest.mark.parametrize("name", ["k", "v", "slots", "positions", "freq"])
@pytest.mark.parametrize("axes,sections,hq", [(1, (64, 0, 0), 4), (3, (16, 24, 24), 2), (0, (0, 0, 0), 4)])
def test_queries_written_over_other_inputs_are_refused(lib, name, axes, sections, hq):
    """At an input's first and last bytes."""
    if axes == 0 and name in ("positions", "freq"):
        return  # not read
    args = dict(tokens=5, axes=axes, sections=sections, hq=hq, q=FAR[0], k=FAR[1], v=FAR[2],
                slots=FAR[3], positions=FAR[4], freq=FAR[5].value, ks=264, vs=512)
    last = dict(k=(4 * 264 + 256) * 2 - 16, v=(4 * 512 + 256) * 2 - 16, slots=32,
                positions=axes * 5 * 4 // 16 * 16, freq=512 - 16)[name]
    base = args[name] if name == "freq" else args[name].value
    for at in (base, base + last, base - (4 * 512 + hq * 128) * 2 + 16):
        assert _append(lib, out=ctypes.c_void_p(at), os=512, **args) == INVALID


def test_keys_within_queries_turned_in_place_are_refused(lib):
    """A key that is a slice of queries that the same call turns in place."""
    args = dict(tokens=3, hq=4, q=FAR[0], out=FAR[0], v=FAR[2], slots=FAR[3], positions=FAR[4],
                freq=FAR[5].value, k=ctypes.c_void_p(FAR[0].value + 512), ks=512)
    assert _append(lib, **args) == INVALID
    args.update(k=FAR[1], v=ctypes.c_void_p(FAR[0].value + 512), vs=512)
    assert _append(lib, **args) == INVALID


APART = dict(tokens=3, hq=4, q=FAR[0], out=ctypes.c_void_p(1 << 44), k=FAR[1], v=FAR[2], slots=FAR[3],
             positions=FAR[4], freq=FAR[5].value)


@pytest.mark.parametrize("kw", [
    dict(v_pages=K), dict(v_pages=K + POOL - 16), dict(k_pages=V + 16), dict(scales=K + POOL - 16),
    dict(scales=K - 8 * 2 * 8 * 4 + 16), dict(scales=V), dict(scales=V + POOL // 2)])
def test_an_append_to_a_cache_whose_arrays_overlap_is_refused(lib, kw):
    assert _append(lib, cache=_cache(**kw), **APART) == INVALID


@pytest.mark.parametrize("name", ["q", "k", "v", "slots", "positions", "freq"])
@pytest.mark.parametrize("begin,size", [(K, POOL), (V, POOL), (S, 8 * 2 * 8 * 4)])
def test_an_append_of_what_lies_in_the_cache_is_refused(lib, name, begin, size):
    least = dict(q=3 * 1024, k=3 * 512, v=3 * 512, slots=24, positions=12, freq=512)[name]
    for at in (begin, begin + size - 16, begin - least // 16 * 16 + 16):
        kw = dict(APART)
        kw[name] = at if name == "freq" else ctypes.c_void_p(at)
        assert _append(lib, **kw) == INVALID


@pytest.mark.parametrize("at,ks,vs", [
    (0, 256, 256), (16, 256, 256), (496, 512, 512), (-496, 512, 512), (1024 - 496, 512, 512),
    (4096 + 496, 512, 512), (2 * 512 * 2, 512, 520)])
def test_keys_and_values_read_over_one_another_are_refused(lib, at, ks, vs):
    """v_out begins `at` bytes behind k_out: five rows of 512 bytes each."""
    batch = dict(num_requests=5, total_q=5)
    assert _read(lib, batch=batch, k=FAR[0], ks=ks, v=ctypes.c_void_p(FAR[0].value + at),
                 vs=vs) == INVALID


@pytest.mark.parametrize("array,size", [("q_offsets", 24), ("seq_lens", 20), ("block_table", 5 * 64 * 4)])
def test_outputs_read_over_the_batch_are_refused(lib, array, size):
    for at in (1 << 40, (1 << 40) + (size - 1) // 16 * 16, (1 << 40) - (4 * 600 + 256) * 2 + 16):
        batch = dict(num_requests=5, total_q=5, q_offsets=1 << 42, seq_lens=1 << 43, block_table=1 << 44)
        batch[array] = 1 << 40
        assert _read(lib, batch=batch, k=ctypes.c_void_p(at), ks=600, v=None) == INVALID
        assert _read(lib, batch=batch, v=ctypes.c_void_p(at), vs=600, k=None) == INVALID
