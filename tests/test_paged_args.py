"""Argument checks of the paged key/value entry points (CPU only: every call
here is refused before anything is launched)."""
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
    c = dsa._CKvCache(8, 2, 128, 0, 4096, 8192, 1.0, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _tables(lib, requests=2, free=FAKE, num_free=8, pages=64, width=4, cap=16, table=FAKE,
            slots=FAKE, positions=FAKE, taken=FAKE, cached=FAKE):
    return lib.dsa_build_tables(requests, cached, FAKE, free, num_free, pages, width, cap, table,
                                FAKE, FAKE, slots, positions, FAKE, taken, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(requests=0), INVALID), (dict(requests=4097), UNSUPPORTED), (dict(num_free=-1), INVALID),
    (dict(free=None), INVALID), (dict(pages=0), INVALID), (dict(width=0), INVALID),
    (dict(cap=-1), INVALID), (dict(table=None), INVALID), (dict(taken=None), INVALID),
    (dict(cached=None), INVALID), (dict(slots=ODD), INVALID), (dict(positions=ODD), INVALID)])
def test_build_tables_refusals(lib, kw, code):
    assert _tables(lib, **kw) == code


def _rope(lib, cache=None, fmt=0, tokens=3, axes=1, sections=(64, 0, 0), freq=4096, positions=FAKE,
          slots=FAKE, hq=4, q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, out=FAKE, os=512):
    import dsa_sparse_attention_step_gb300 as dsa
    r = dsa._CRope(axes, (ctypes.c_int32 * 3)(*sections), 0, freq)
    c = _cache() if cache is None else cache
    return lib.dsa_rope_append(tokens, ctypes.byref(c), fmt, ctypes.byref(r), positions, slots, hq,
                               q, qs, k, ks, v, vs, out, os, None, None)


CACHE_REFUSALS = [
    (dict(head_dim=96), UNSUPPORTED), (dict(format=1), UNSUPPORTED), (dict(format=7), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_pages=1 << 20, num_kv_heads=1 << 11), INVALID), (dict(k_pages=0), INVALID),
    (dict(v_pages=8200), INVALID), (dict(k_scale=0.5), INVALID),
    (dict(format=2, k_scale=0.0), INVALID), (dict(format=2, v_scale=float("inf")), INVALID),
    (dict(format=2, k_scale=float("nan")), INVALID)]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_cache_refusals_by_rope_append(lib, kw, code):
    assert _rope(lib, cache=_cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(axes=4), UNSUPPORTED),
    (dict(axes=-1), UNSUPPORTED), (dict(sections=(-8, 0, 0)), INVALID),
    (dict(sections=(72, 0, 0)), INVALID), (dict(sections=(12, 0, 0)), UNSUPPORTED),
    (dict(freq=0), INVALID), (dict(positions=None), INVALID), (dict(slots=None), INVALID),
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(qs=516), INVALID),
    (dict(qs=504), INVALID), (dict(ks=248), INVALID), (dict(vs=260), INVALID), (dict(k=ODD), INVALID),
    (dict(out=None), INVALID), (dict(os=500), INVALID), (dict(hq=-1), INVALID),
    (dict(hq=1 << 15, qs=1 << 22, os=1 << 22), UNSUPPORTED)])
def test_rope_append_refusals(lib, kw, code):
    assert _rope(lib, **kw) == code


def test_rope_append_of_no_tokens_is_a_no_op(lib):
    assert _rope(lib, tokens=0) == 0


def _attention(lib, batch=None, cache=None, fmt=0, hq=4, q=FAKE, qs=512, sm=0.1, out=FAKE, ws=FAKE,
               ws_bytes=1 << 40):
    import dsa_sparse_attention_step_gb300 as dsa
    b = dsa._CBatch(1, 1, 1, 4096, 8, 64, 64, 16, 32, 48)
    for k, v in (batch or {}).items():
        setattr(b, k, v)
    c = _cache() if cache is None else cache
    return lib.dsa_paged_attention(ctypes.byref(b), ctypes.byref(c), fmt, hq, q, qs, sm, out, None,
                                   ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_cache_refusals_by_paged_attention(lib, kw, code):
    assert _attention(lib, cache=_cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=dict(page_size=32)), UNSUPPORTED), (dict(batch=dict(max_pages=10)), INVALID),
    (dict(batch=dict(num_pages=9)), INVALID), (dict(fmt=1), UNSUPPORTED), (dict(hq=0), INVALID),
    (dict(hq=5), INVALID), (dict(hq=1 << 15, qs=1 << 22), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(q=ODD), INVALID), (dict(qs=500), INVALID), (dict(sm=0.0), INVALID),
    (dict(sm=float("nan")), INVALID), (dict(sm=float("inf")), INVALID), (dict(out=None), INVALID),
    (dict(out=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=ODD), WORKSPACE),
    (dict(ws_bytes=1000), WORKSPACE),
    # 2^20 new tokens of one request, each over up to 2^20 positions
    (dict(batch=dict(total_q=1 << 20, max_q_per_request=1 << 20, max_seq_len=1 << 20,
                     max_pages=1 << 14)), UNSUPPORTED)])
def test_paged_attention_refusals(lib, kw, code):
    assert _attention(lib, **kw) == code


def test_paged_attention_of_no_tokens_is_a_no_op(lib):
    assert _attention(lib, batch=dict(total_q=0), q=None, out=None, ws=None) == 0


def test_paged_attention_workspace_follows_rows_and_head_dim(lib):
    import dsa_sparse_attention_step_gb300 as dsa
    b = dsa._CBatch(4, 4, 1, 4096, 8, 64, 64, 16, 32, 48)

    def size(hq, **kw):
        c = _cache(**kw)
        return lib.dsa_paged_attention_workspace_size(ctypes.byref(b), ctypes.byref(c), hq)
    assert 0 < size(4) == size(32) < size(64) < size(80) == size(96) < size(128) == size(256)
    # 256 dims have no tile of 48 rows: 40 rows take the 64-row one
    assert size(80, head_dim=256) == size(128, head_dim=256)
    assert size(4, head_dim=256) > size(4) > size(4, head_dim=64)
    assert size(5) == 0 and size(0) == 0 and size(4, head_dim=96) == 0


# Arrays of a call for 2 requests, 8 free pages, 4 table columns and 16 tokens, apart.
TABLE_ARRAYS = dict(cached=(4096, 8), new=(8192, 8), free=(12288, 32), table=(16384, 32),
                    q_offsets=(20480, 12), seq_lens=(24576, 8), slots=(28672, 128),
                    positions=(32768, 64), requests=(36864, 64), taken=(40960, 4),
                    status=(45056, 4))
TABLE_INPUTS = ("cached", "new", "free")


@pytest.mark.parametrize("name", [n for n in TABLE_ARRAYS if n not in TABLE_INPUTS])
@pytest.mark.parametrize("other", list(TABLE_ARRAYS))
def test_build_tables_refuses_an_output_that_overlaps(lib, name, other):
    """In place (seq_lens as cached_lens), whole or by an edge: CTAs would read what
    others write."""
    if name == other:
        return
    at, size = TABLE_ARRAYS[other]
    own = TABLE_ARRAYS[name][1]
    ends = [at] if name in ("slots", "positions", "requests") else [at, at + size - 4,
                                                                    at - own + 4]
    for begin in ends:
        a = {n: ctypes.c_void_p(begin if n == name else TABLE_ARRAYS[n][0]) for n in TABLE_ARRAYS}
        assert lib.dsa_build_tables(2, a["cached"], a["new"], a["free"], 8, 64, 4, 16, a["table"],
                                    a["q_offsets"], a["seq_lens"], a["slots"], a["positions"],
                                    a["requests"], a["taken"], a["status"], None) == INVALID


@pytest.mark.parametrize("sm,k_scale", [(1e-25, 1e-25), (1e30, 1e30), (1e-38, 1e-3)])
def test_paged_attention_refuses_score_factors_outside_fp32(lib, sm, k_scale):
    assert _attention(lib, cache=_cache(format=2, k_scale=k_scale), sm=sm) == INVALID
