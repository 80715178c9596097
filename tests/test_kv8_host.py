"""The 8-bit K/V cache operators without a GPU: refusals that come before any launch, the index arithmetic of the
kernels (csrc/kv8_map.h, compiled here) against counting, and the oracle's own rounding."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import kv8
from quantized_decode_gb300 import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that is aligned and never used: every call below returns before it could be


@pytest.fixture(scope="module")
def lib():
    import quantized_decode_gb300 as qd
    qd.build()
    return qd.load()


GOOD = dict(format=1, n_kv_heads=4, head_dim=128, n_pool_pages=10, k_codes=P, v_codes=P, k_scale=P, v_scale=P, page_table=P,
            n_seqs=2, table_stride=5)
BAD_CACHES = [dict(format=0), dict(format=3), dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(head_dim=96), dict(head_dim=256),
              dict(n_pool_pages=0), dict(n_pool_pages=1 << 25), dict(k_codes=None), dict(v_codes=P + 8), dict(k_scale=P + 2),
              dict(v_scale=None), dict(page_table=P + 1), dict(n_seqs=0), dict(n_seqs=4097), dict(table_stride=0),
              dict(table_stride=1 << 27)]


def _cache(**kw):
    return ctypes.byref(L.llm_kv8_cache(**{**GOOD, **kw}))


ROWS = dict(dtype=0, k=P, ks=512, v=P, vs=512, rs=P, kv=P, n=3, err=P)
BAD_ROWS = [dict(dtype=3), dict(dtype=-1), dict(k=None), dict(k=P + 4), dict(ks=511), dict(ks=514), dict(ks=0), dict(ks=-512),
            dict(v=P + 8), dict(vs=500), dict(rs=None), dict(rs=P + 2), dict(kv=None), dict(n=0), dict(n=-5), dict(err=P + 1),
            dict(dtype=1, ks=516)]


@pytest.mark.parametrize("name", ["append", "read"])
def test_row_calls_refuse(lib, name):
    def call(cache=None, **kw):
        a = {**ROWS, **kw}
        cache = _cache() if cache is None else cache
        if name == "append":
            return lib.llm_op_kv8_append(cache, a["dtype"], a["k"], a["ks"], a["v"], a["vs"], a["rs"], a["kv"], a["n"], a["err"], None)
        return lib.llm_op_kv8_read(cache, a["dtype"], a["rs"], a["kv"], a["n"], a["k"], a["ks"], a["v"], a["vs"], a["err"], None)

    assert lib.llm_op_kv8_append(None, 0, P, 512, P, 512, P, P, 1, P, None) == L.LLM_ERR_ARG
    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == L.LLM_ERR_ARG, bad
    for bad in BAD_ROWS:
        assert call(**bad) == L.LLM_ERR_ARG, bad


def test_attention_refuses(lib):
    good = dict(dtype=0, q=P, qs=28 * 128, rs=P, kv=P, n=3, hq=28, out=P, lse=P, ws=P, wb=1 << 40, err=P)

    def call(cache=None, **kw):
        a = {**good, **kw}
        return lib.llm_op_kv8_attention(_cache() if cache is None else cache, a["dtype"], a["q"], a["qs"], a["rs"], a["kv"], a["n"],
                                        a["hq"], a["out"], a["lse"], a["ws"], a["wb"], a["err"], None)

    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == L.LLM_ERR_ARG, bad
    for bad in (dict(dtype=7), dict(q=None), dict(q=P + 8), dict(qs=28 * 128 - 4), dict(qs=28 * 128 + 2), dict(rs=None), dict(kv=P + 2),
                dict(n=0), dict(hq=0), dict(hq=30), dict(hq=36), dict(hq=-4), dict(out=None), dict(out=P + 4), dict(lse=P + 1),
                dict(ws=None), dict(ws=P + 128), dict(err=P + 3)):
        assert call(**bad) == L.LLM_ERR_ARG, bad
    need = ctypes.c_int64()
    for cache, hq, n in ((_cache(head_dim=1), 4, 1), (_cache(), 30, 1), (_cache(), 36, 1), (_cache(), 4, 0)):
        assert lib.llm_op_kv8_attention_workspace(cache, hq, n, ctypes.byref(need)) == L.LLM_ERR_ARG
    assert lib.llm_op_kv8_attention_workspace(_cache(), 28, 1, None) == L.LLM_ERR_ARG


def test_rope_refuses(lib):
    good = dict(dtype=0, q=P, qs=1024, k=P, ks=1024, gq=P, gk=P, eps=1e-6, base=1e6, pos=P, n=2, hq=8, hkv=2, d=128, qo=P, ko=P)

    def call(**kw):
        return lib.llm_op_qk_norm_rope(*{**good, **kw}.values(), None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(dtype=3), dict(q=None), dict(q=P + 4), dict(qs=1020), dict(qs=1026), dict(ks=250), dict(gq=None), dict(gk=None),
                dict(gq=P + 2), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(base=0.0), dict(base=-1.0), dict(base=nan),
                dict(base=inf), dict(pos=None), dict(pos=P + 2), dict(n=0), dict(hq=0), dict(hkv=0), dict(d=32), dict(d=256),
                dict(qo=None), dict(ko=P + 8), dict(hq=70000, qs=1 << 30)):
        assert call(**bad) == L.LLM_ERR_ARG, bad


# ---------------------------------------------------------------- index arithmetic

MAIN = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include "kv8_map.h"
using namespace qd;
static unsigned long long st = 12345;
static int rnd(int n) { st = st * 6364136223846793005ull + 1442695040888963407ull; return (int)((st >> 33) % (unsigned)n); }
#define CHECK(c) do { if (!(c)) { printf("failed: %s, line %d, trial %d\n", #c, __LINE__, trial); return 1; } } while (0)
int main() {
    for (int trial = 0; trial < 4000; ++trial) {
        // sequences with any numbers in their range: every (row, token) is met exactly once, and nothing else
        const int B = 1 + rnd(40), stride = 1 + rnd(8);
        int start[42], kv[41], n_rows;
        start[0] = rnd(3);
        for (int b = 0; b < B; ++b) {
            kv[b] = rnd(stride * 16 + 1);
            const int n = rnd(4) == 0 ? 0 : (rnd(2) ? rnd(kv[b] + 1) : (kv[b] > 0));
            start[b + 1] = start[b] + n;
        }
        n_rows = start[B] + rnd(3);
        if (n_rows < 1) n_rows = 1;
        const bool wild = trial % 4 == 3;  // numbers out of range: nothing outside the arrays
        if (wild)
            for (int i = 0; i < 3; ++i) {
                const int junk[6] = {-5, 1 << 30, -2147483647 - 1, 2147483647, n_rows + 1, 0};
                if (rnd(2)) start[rnd(B + 1)] = junk[rnd(6)];
                else kv[rnd(B)] = junk[rnd(6)];
            }
        static int met[16384];
        memset(met, 0, sizeof met);
        const long long items = kv8_items(n_rows, B);
        for (long long it = 0; it < items; ++it) {
            int b = 0;  // the last sequence whose items begin at or before `it`
            for (int i = 0; i < B; ++i)
                if (kv8_item_base(start[i], i) <= it) b = i;
            const Kv8Seq s = kv8_seq(start[b], start[b + 1], kv[b], n_rows, stride);
            const Kv8Span p = kv8_span(s, it - kv8_item_base(start[b], b));
            if (p.count == 0) continue;
            CHECK(p.count > 0 && p.slot0 >= 0 && p.slot0 + p.count <= 16 && p.page >= 0 && p.page < stride);
            CHECK(p.row0 >= 0 && p.row0 + p.count <= n_rows);
            for (int i = 0; i < p.count; ++i) {
                if (!wild) {
                    CHECK(p.row0 + i >= start[b] && p.row0 + i < start[b + 1]);
                    CHECK(p.page * 16 + p.slot0 + i == kv[b] - (start[b + 1] - start[b]) + p.row0 + i - start[b]);
                }
                ++met[p.row0 + i];
            }
        }
        if (!wild)
            for (int r = 0; r < n_rows; ++r) CHECK(met[r] == (r >= start[0] && r < start[B]));
        // attention: pages and blocks within the table, for every length that it can hold
        for (int b = 0; b < B; ++b) {
            const Kv8Seq s = kv8_seq(start[b], start[b + 1], kv[b], n_rows, stride);
            CHECK(s.row0 >= 0 && s.rows >= 0 && s.row0 + s.rows <= n_rows);
            const int kvb = s.kv < 0 || s.kv > stride * 16 ? 0 : s.kv;
            CHECK(kv8_pages(kvb) >= 1 && kv8_pages(kvb) <= stride);
        }
        const int most = 2147483647 - 15;  // 2^27 - 1 pages
        const int left = trial < 300 ? trial : (trial < 600 ? most - (trial - 300) : rnd(most + 1));
        const long long nb = kv8_blocks(left, 128);
        CHECK(nb * 128 >= left && (nb - 1) * 128 < left + (left == 0));
        for (long long p = nb * 8 - 9; p < nb * 8; ++p)
            if (p >= 0) CHECK(kv8_page_there((int)p, left) == (p * 16 < left));
        CHECK(left == 0 || (long long)kv8_pages(left) * 16 >= left);
    }
    printf("ok\n");
    return 0;
}
"""


def test_index_arithmetic(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "map.cpp", tmp_path / "map"
    src.write_text(MAIN)
    subprocess.check_call([cc, "-std=c++17", "-O1", "-fsanitize=undefined,address", "-I",
                           os.path.join(ROOT, "quantized_decode_gb300", "csrc"), str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


# ---------------------------------------------------------------- the oracle's rounding


def test_e4m3_codes_round_trip_and_nearest():
    torch = pytest.importorskip("torch")
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    np.testing.assert_array_equal(kv8.encode(kv8.decode(codes, "e4m3"), "e4m3"), codes)
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.float32(2.0) ** np.random.default_rng(1).integers(-12, 9, 20000)
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(kv8.encode(x, "e4m3"), want)


def test_append_keeps_values_within_half_a_step():
    """Rows written at once: |value - x| <= scale / 2 (int8), 2^-4 of |x| or 2^-10 of the scale (e4m3)."""
    rng = np.random.default_rng(2)
    for fmt in ("int8", "e4m3"):
        cache = {"fmt": fmt, "k": np.zeros((4, 2, 16, 64), np.uint8), "v": np.zeros((4, 2, 16, 64), np.uint8),
                 "ks": np.zeros((4, 2), np.float32), "vs": np.zeros((4, 2), np.float32)}
        table = np.array([[2, 0, 1]], np.int32)
        x = rng.standard_normal((2, 40, 2, 64)).astype(np.float32)
        kv8.append(cache, table, [0, 40], [40], x[0], x[1])
        k, v = kv8.read(cache, table, [0, 40], [40], 40)
        for got, want, s in ((k, x[0], cache["ks"]), (v, x[1], cache["vs"])):
            step = s[table[0]][np.arange(40) // 16][:, :, None]
            tol = step * 0.5 if fmt == "int8" else np.maximum(np.abs(want) * 2.0 ** -4, step * 2.0 ** -10)
            assert np.all(np.abs(got - want) <= tol * 1.0001)
