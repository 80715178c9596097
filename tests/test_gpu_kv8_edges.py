"""The 8-bit K/V cache operators where they are easily wrong: V scales so far apart that sums are rescaled again and
again, blocks that are not finite, sequences whose numbers are out of order, calls after one that failed
(GPU required).  The definitions in 64 bits are oracle/kv8.py's."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8
from quantized_decode_gb300 import _lib as L

from ._kv8 import DTYPES, DeviceCache, as_f32, attention_bounds, host_cache, ints, page_table, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    L.load()


def _rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DTYPES[dtype][0]).cuda()


def _call(dev, dtype, q, rows, kv):
    out = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 55.0, device="cuda")
    assert dev.attention(dtype, q, ints(starts(rows)), ints(kv), out, lse) == 0
    torch.cuda.synchronize()
    assert dev.err.item() == 0
    return as_f32(out), lse.cpu().numpy()


def _bounds(dtype, ref, kv):
    """attention_bounds, with the smallest weights where V scales differ: a weight is kept as fp16 of its size times the
    page's V scale over the reference one, 2^-4 to 2^4, next to a largest of 2^7: fp16's 2^-25 below its
    normal numbers is 2^-25 2^4 2^-7 = 2^-28 of the largest weight, whatever the row type."""
    tol, ltol = attention_bounds(dtype, *ref, kv)
    return tol + ref[3] * 2.0 ** -28, ltol


# ---------------------------------------------------------------- rows of fp16


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (7, 1, 128), (2, 2, 128)])
@pytest.mark.parametrize("rows,kv", [((1, 1), (20000, 333)), ((1,), (3000,)), ((4, 3), (3000, 64)), ((12, 9), (3000, 64)), ((6,), (9000,))])
def test_fp16_steps_and_drafts_are_as_exact_as_their_rounding(fmt, Hq, Hkv, d, rows, kv):
    """Weights of 11 bits would be off by as much as the rounding of the result: both products have to be as those of
    fp32 rows, and the result half a step off (2^-11 of it, 2^-25 among the numbers below 2^-14)."""
    rng = np.random.default_rng(50)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, fmt, pages, Hkv, d)
    q = _rand(rng, (sum(rows), Hq, d), "f16", 2.0)
    out, lse = _call(DeviceCache(host, table), "f16", q, rows, kv)
    ref = kv8.attention(host, table, starts(rows), kv, as_f32(q))
    tol, ltol = _bounds("f32", ref, max(kv))
    off = np.abs(out - ref[0]) / (tol + np.abs(ref[0]) * 2.0 ** -11 + 2.0 ** -25)
    assert np.all(off <= 1), (float(off.max()), float(np.mean(off > 1)))
    assert np.all(np.abs(lse - ref[1]) <= ltol)
