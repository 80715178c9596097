"""The 16-bit K/V cache operators without a GPU: refusals that come before any launch, and the oracle's own choice of slots."""
import ctypes

import numpy as np
import pytest

from oracle import kv16
from quantized_decode_gb300 import _lib as L

P = 1 << 20  # an address that is aligned and never used: every call below returns before it could be


@pytest.fixture(scope="module")
def lib():
    import quantized_decode_gb300 as qd
    qd.build()
    return qd.load()


GOOD = dict(dtype=2, n_kv_heads=4, head_dim=128, n_pool_pages=10, k_pool=P, v_pool=P, page_table=P, n_seqs=2, table_stride=5)
BAD_CACHES = [dict(dtype=0), dict(dtype=3), dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(head_dim=96), dict(head_dim=256),
              dict(n_pool_pages=0), dict(n_pool_pages=1 << 25), dict(k_pool=None), dict(v_pool=P + 8), dict(page_table=P + 1),
              dict(page_table=None), dict(n_seqs=0), dict(n_seqs=4097), dict(table_stride=0), dict(table_stride=1 << 27)]
PREFIX = dict(page_table=P, len=P, seq_start=P, n_groups=2, table_stride=3)
BAD_PREFIXES = [dict(page_table=None), dict(len=P + 1), dict(len=None), dict(seq_start=P + 2), dict(n_groups=0), dict(n_groups=4097),
                dict(table_stride=0), dict(table_stride=1 << 27)]


def _cache(**kw):
    return ctypes.byref(L.llm_kv16_cache(**{**GOOD, **kw}))


def _prefix(**kw):
    return ctypes.byref(L.llm_kv16_prefix(**{**PREFIX, **kw}))


def test_rope_append_refuses(lib):
    axis = (ctypes.c_uint8 * 64)(*[i % 3 for i in range(64)])
    far = (ctypes.c_uint8 * 64)(*[3 if i == 63 else 0 for i in range(64)])
    good = dict(dtype=0, q=P, qs=28 * 128, k=P, ks=512, v=P, vs=512, qg=None, kg=None, eps=1e-6, base=1e6, axis=axis, na=3, pos=P, rs=P, kv=P,
                n=3, hq=28, out=P, err=P)

    def call(cache=None, **kw):
        a = {**good, **kw}
        return lib.llm_op_kv16_rope_append(_cache() if cache is None else cache, a["dtype"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                                           a["qg"], a["kg"], a["eps"], a["base"], a["axis"], a["na"], a["pos"], a["rs"], a["kv"], a["n"],
                                           a["hq"], a["out"], a["err"], None)

    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == L.LLM_ERR_ARG, bad
    for bad in (dict(dtype=3), dict(q=None), dict(q=P + 8), dict(qs=28 * 128 - 4), dict(qs=28 * 128 + 2), dict(k=P + 4), dict(ks=500), dict(v=None),
                dict(vs=514), dict(qg=P), dict(kg=P), dict(qg=P + 2, kg=P), dict(eps=-1.0), dict(eps=float("nan")), dict(base=0.0),
                dict(base=float("inf")), dict(axis=None), dict(axis=far), dict(na=0), dict(na=9), dict(na=2), dict(pos=None), dict(pos=P + 2),
                dict(rs=P + 1), dict(kv=None), dict(n=0), dict(hq=0), dict(hq=65537), dict(out=P + 8), dict(err=P + 1), dict(dtype=1, ks=516)):
        assert call(**bad) == L.LLM_ERR_ARG, bad


def test_attention_refuses(lib):
    good = dict(q=P, qs=28 * 128, rs=P, kv=P, n=3, hq=28, out=P, lse=P, ws=P, wb=1 << 40, err=P)

    def call(cache=None, prefix=None, **kw):
        a = {**good, **kw}
        return lib.llm_op_kv16_attention(_cache() if cache is None else cache, prefix, a["q"], a["qs"], a["rs"], a["kv"], a["n"], a["hq"],
                                         a["out"], a["lse"], a["ws"], a["wb"], a["err"], None)

    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == L.LLM_ERR_ARG, bad
    for bad in BAD_PREFIXES:
        assert call(None, _prefix(**bad)) == L.LLM_ERR_ARG, bad
    for bad in (dict(q=None), dict(q=P + 8), dict(qs=28 * 128 - 8), dict(qs=28 * 128 + 4), dict(rs=None), dict(kv=P + 2), dict(n=0), dict(hq=0),
                dict(hq=30), dict(hq=36), dict(hq=-4), dict(out=None), dict(out=P + 4), dict(lse=P + 1), dict(ws=None), dict(ws=P + 128),
                dict(err=P + 2)):
        assert call(**bad) == L.LLM_ERR_ARG, bad
    need = ctypes.c_int64()
    for bad in BAD_CACHES:
        assert lib.llm_op_kv16_attention_workspace(_cache(**bad), None, 28, 1, ctypes.byref(need)) == L.LLM_ERR_ARG
    for bad in BAD_PREFIXES:
        assert lib.llm_op_kv16_attention_workspace(_cache(), _prefix(**bad), 28, 1, ctypes.byref(need)) == L.LLM_ERR_ARG
    for hq, n in ((27, 1), (0, 1), (36, 1), (28, 0)):
        assert lib.llm_op_kv16_attention_workspace(_cache(), None, hq, n, ctypes.byref(need)) == L.LLM_ERR_ARG
    assert lib.llm_op_kv16_attention_workspace(_cache(), None, 28, 1, None) == L.LLM_ERR_ARG


def test_weigh_refuses(lib):
    good = dict(q=P, qs=28 * 128, rs=P, kv=P, n=3, hq=28, lse=P, keep=1.0, s=P, ss=100, err=P)

    def call(cache=None, **kw):
        a = {**good, **kw}
        return lib.llm_op_kv16_weigh(_cache() if cache is None else cache, a["q"], a["qs"], a["rs"], a["kv"], a["n"], a["hq"], a["lse"],
                                     a["keep"], a["s"], a["ss"], a["err"], None)

    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == L.LLM_ERR_ARG, bad
    for bad in (dict(q=P + 2), dict(qs=100), dict(rs=None), dict(kv=P + 1), dict(n=-1), dict(hq=3), dict(hq=64), dict(lse=None), dict(lse=P + 2),
                dict(keep=-0.5), dict(keep=float("nan")), dict(keep=float("inf")), dict(s=None), dict(s=P + 2), dict(ss=0), dict(err=P + 3)):
        assert call(**bad) == L.LLM_ERR_ARG, bad


def test_evict_refuses(lib):
    good = dict(kv=P, budget=64, first=4, last=16, s=P, so=P, ss=100, kept=P, new=2 * P, err=P)

    def call(cache=None, **kw):
        a = {**good, **kw}
        return lib.llm_op_kv16_evict(_cache() if cache is None else cache, a["kv"], a["budget"], a["first"], a["last"], a["s"], a["so"], a["ss"],
                                     a["kept"], a["new"], a["err"], None)

    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == L.LLM_ERR_ARG, bad
    for bad in (dict(kv=None), dict(budget=0), dict(first=-1), dict(last=-1), dict(first=60), dict(first=2**31 - 1, last=2**31 - 1), dict(s=None),
                dict(so=P + 2), dict(ss=63), dict(kept=None), dict(new=P), dict(new=None), dict(err=P + 1)):
        assert call(**bad) == L.LLM_ERR_ARG, bad


def test_choice_of_slots():
    s = np.array([9, 1, 5, np.nan, 5, -0.0, 0.0, 5, -np.inf, 2, 3], np.float32)
    assert kv16.choose(s, 11, 6, 1, 2).tolist() == [0, 2, 4, 7, 9, 10]
    assert kv16.choose(s, 11, 5, 1, 2).tolist() == [0, 2, 4, 9, 10]      # the lower slot of those alike
    assert kv16.choose(s, 11, 8, 1, 2).tolist() == [0, 1, 2, 4, 5, 7, 9, 10]
    assert kv16.choose(s, 11, 10, 1, 2).tolist() == [0, 1, 2, 4, 5, 6, 7, 8, 9, 10]  # the NaN goes first of all
    assert kv16.choose(s, 11, 3, 1, 2).tolist() == [0, 9, 10]
    assert kv16.choose(s, 4, 4, 1, 2).tolist() == [0, 1, 2, 3]
