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


# ---------------------------------------------------------------- V scales far apart


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 4, 12])
def test_a_tiny_scale_after_many_large_ones(fmt, dtype, rows):
    """Every warp goes through two pages of scale 1, eighty or more of scale 15 whose codes are the largest and of one sign
    in each dim, and then pages of 2^-110: the sum so far must not leave fp32's range when its unit moves.  20
    sequences of 8 heads, so that no segment is cut: its 1008 pages go round the 8 or 12 warps of one CTA."""
    rng = np.random.default_rng(51)
    n, Hkv, d, pages = 20, 8, 64, 1008
    sign = np.where(rng.random((Hkv, 1, d)) < 0.5, -1, 1)
    v = np.broadcast_to(sign * float(kv8.CODE_MAX[fmt]), (pages, Hkv, 16, d)).astype(np.float32)
    host = host_cache(rng, fmt, pages, Hkv, d)
    host["v"] = kv8.encode(v, fmt)
    host["ks"][:] *= np.float32(2.0 ** -6)  # near even weights
    host["vs"][:24], host["vs"][24:-24], host["vs"][-24:] = 1, 15, np.float32(2.0 ** -110)
    table = np.broadcast_to(np.arange(pages, dtype=np.int32), (n, pages))
    q = _rand(rng, (rows, Hkv, d), dtype)
    out, lse = _call(DeviceCache(host, table), dtype, q.repeat(n, 1, 1), (rows,) * n, (16 * pages,) * n)
    ref = kv8.attention(host, table, [0, rows], [16 * pages], as_f32(q))
    tol, ltol = _bounds(dtype, ref, 16 * pages)
    for i in range(n):
        assert np.all(np.abs(out[i * rows:(i + 1) * rows] - ref[0]) <= tol)
        assert np.all(np.abs(lse[i * rows:(i + 1) * rows] - ref[1]) <= ltol)


@pytest.mark.parametrize("fmt,dtype", [("int8", "f32"), ("e4m3", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("rows", [1, 12])
@pytest.mark.parametrize("spread", [3, 10, 40])
def test_scales_far_apart_in_long_sequences(fmt, dtype, rows, spread):
    """Dozens of pages to a warp, whose V scales wander by up to 2^(2 spread), with zeros and missing K scales."""
    rng = np.random.default_rng(52 + spread)
    n, Hkv, d, pages = 8, 4, 64, 1200
    host = host_cache(rng, fmt, pages, Hkv, d)
    host["vs"] *= np.float32(2.0) ** rng.integers(-spread, spread + 1, host["vs"].shape).astype(np.float32)
    host["vs"][rng.random(host["vs"].shape) < 0.05] = 0
    host["ks"][rng.random(host["ks"].shape) < 0.05] = 0
    table = np.stack([rng.permutation(pages).astype(np.int32) for _ in range(n)])
    kv = tuple(int(x) for x in rng.integers(12000, 16 * pages + 1, n))
    q = _rand(rng, (n * rows, Hkv, d), dtype, 0.5)
    if dtype == "f16":  # outputs within fp16's range
        host["vs"] *= np.float32(2.0 ** -(spread + 6))
    out, lse = _call(DeviceCache(host, table), dtype, q, (rows,) * n, kv)
    ref = kv8.attention(host, table, starts((rows,) * n), kv, as_f32(q))
    tol, ltol = _bounds(dtype, ref, max(kv))
    assert np.all(np.abs(out - ref[0]) <= tol), float((np.abs(out - ref[0]) / tol).max())
    assert np.all(np.abs(lse - ref[1]) <= ltol)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [1, 12, 150])
def test_small_weights_at_small_scales(fmt, dtype, rows):
    """V scales just above 1/16 of the first page's, so that the unit stays, and weights down to 2^-24 of the largest."""
    rng = np.random.default_rng(53)
    Hkv, d, pages = 2, 64, 400
    table, total = page_table(rng, [16 * pages])
    host = host_cache(rng, fmt, total, Hkv, d)
    host["vs"][:] = np.float32(1 / 15.9)
    host["vs"][table[0, :64]] = 1
    q = _rand(rng, (rows, Hkv, d), dtype, 2.0)
    out, lse = _call(DeviceCache(host, table), dtype, q, (rows,), (16 * pages,))
    ref = kv8.attention(host, table, [0, rows], [16 * pages], as_f32(q))
    tol, ltol = _bounds(dtype, ref, 16 * pages)
    assert np.all(np.abs(out - ref[0]) <= tol)
    assert np.all(np.abs(lse - ref[1]) <= ltol)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (2, 1, 128)])
@pytest.mark.parametrize("rows,kv", [((1,), (300,)), ((1, 1), (9000, 40)), ((12,), (700,)), ((200,), (300,)), ((120,), (4000,))])
def test_v_near_the_smallest_numbers(Hq, Hkv, d, rows, kv):
    """V of about 2^-118 keeps its bits: results scale with V as they do in 64 bits, but for the steps of 2^-149 that fp32
    has near 0 (one rounding in each warp, part and row)."""
    rng = np.random.default_rng(59)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "int8", pages, Hkv, d)
    q = _rand(rng, (sum(rows), Hq, d), "f32", 2.0)
    ref = kv8.attention(host, table, starts(rows), kv, as_f32(q))
    tol, ltol = _bounds("f32", ref, max(kv))
    host["vs"] *= np.float32(2.0 ** -118)
    out, lse = _call(DeviceCache(host, table), "f32", q, rows, kv)
    assert np.all(np.abs(out.astype(np.float64) * 2.0 ** 118 - ref[0]) <= tol + 4 * 2.0 ** (118 - 149))
    assert np.all(np.abs(lse - ref[1]) <= ltol)


# ---------------------------------------------------------------- blocks that are not finite

NAN_CALLS = {  # rows, length, capacity of the table
    "step": (1, 300, 300),
    "draft": (4, 300, 300),
    "long draft": (30, 300, 300),
    "prompt": (200, 300, 300),
    "prompt of few rows over many keys": (120, 3000, 5008),
}


@pytest.mark.parametrize("fmt,dtype", [("e4m3", "f32"), ("int8", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (2, 2, 128)])
@pytest.mark.parametrize("call", list(NAN_CALLS))
def test_a_nan_block_of_v_leaves_lse_alone(fmt, dtype, Hq, Hkv, d, call):
    """V's scale has no part in lse: where it is NaN, out is NaN for the rows that see the block, and lse stays what q and
    K make it."""
    rng = np.random.default_rng(54)
    rows, kv, most = NAN_CALLS[call]
    table, pages = page_table(rng, [kv], capacity=[most])
    host = host_cache(rng, fmt, pages, Hkv, d)
    q = _rand(rng, (rows, Hq, d), dtype, 2.0)
    ref = kv8.attention(host, table, [0, rows], [kv], as_f32(q))
    tol, ltol = _bounds(dtype, ref, kv)
    for page in (0, (kv - rows // 2 - 1) // 16, (kv - 1) // 16):
        bad = {**host, "vs": host["vs"].copy()}
        bad["vs"][table[0, page], 1] = np.nan
        out, lse = _call(DeviceCache(bad, table), dtype, q, (rows,), (kv,))
        hit = np.zeros((rows, Hq), bool)
        hit[max(0, 16 * page - (kv - rows)):, Hq // Hkv:] = True
        assert np.all(np.isnan(out[hit])) and np.all((np.abs(out - ref[0]) <= tol)[~hit])
        assert np.all(np.abs(lse - ref[1]) <= ltol)


@pytest.mark.parametrize("rows", [1, 12, 200])
def test_nothing_but_nan_and_zero_blocks_of_v(rows):
    """No V scale that could be a unit: all of them NaN or 0, in one order and the other."""
    rng = np.random.default_rng(55)
    Hq, Hkv, d, kv = 4, 2, 64, 260
    table, pages = page_table(rng, [kv])
    host = host_cache(rng, "int8", pages, Hkv, d)
    q = _rand(rng, (rows, Hq, d), "f32", 2.0)
    for pattern in (lambda p: np.nan, lambda p: np.nan if p < 8 else 0.0, lambda p: 0.0 if p < 8 else np.nan,
                    lambda p: np.nan if p == 0 else 1e-30):
        host["vs"][table[0]] = np.array([pattern(p) for p in range(table.shape[1])], np.float32)[:, None]
        out, lse = _call(DeviceCache(host, table), "f32", q, (rows,), (kv,))
        with np.errstate(invalid="ignore"):
            ref = kv8.attention(host, table, [0, rows], [kv], as_f32(q))
        ltol = _bounds("f32", ref, kv)[1]
        np.testing.assert_array_equal(np.isnan(out), np.isnan(ref[0]))
        fine = ~np.isnan(ref[0])
        assert np.all(out[fine] == 0) and np.all(ref[0][fine] == 0)
        assert np.all(np.abs(lse - ref[1]) <= ltol)


@pytest.mark.parametrize("rows", [1, 12, 200])
def test_a_nan_block_of_k_makes_nan_of_out_and_lse(rows):
    rng = np.random.default_rng(56)
    Hq, Hkv, d, kv = 4, 2, 64, 300
    table, pages = page_table(rng, [kv])
    host = host_cache(rng, "int8", pages, Hkv, d)
    q = _rand(rng, (rows, Hq, d), "f32", 2.0)
    ref = kv8.attention(host, table, [0, rows], [kv], as_f32(q))
    tol, ltol = _bounds("f32", ref, kv)
    page = (kv - rows // 2 - 1) // 16
    host["ks"][table[0, page], 0] = np.nan
    out, lse = _call(DeviceCache(host, table), "f32", q, (rows,), (kv,))
    hit = np.zeros((rows, Hq), bool)
    hit[max(0, 16 * page - (kv - rows)):, :Hq // Hkv] = True
    assert np.all(np.isnan(out[hit])) and np.all(np.isnan(lse[hit]))
    assert np.all((np.abs(out - ref[0]) <= tol)[~hit]) and np.all((np.abs(lse - ref[1]) <= ltol)[~hit])


# ---------------------------------------------------------------- numbers out of order, calls after a failure

FALLING = {  # row_start with a sequence that ends before it begins, no work item of which there is
    "3 sequences": [0, 64, 32, 64],
    "40 sequences": [0, 64, 32] + list(range(64, 102)),
    "a prompt among 3": [0, 512, 300, 600],
    "a prompt among 40": [0, 2560, 2304] + list(range(2600, 2638)),
}


@pytest.mark.parametrize("call", list(FALLING))
def test_row_starts_that_fall_are_reported(call):
    rng = np.random.default_rng(57)
    rs = FALLING[call]
    n, B, Hkv, d = rs[-1], len(rs) - 1, 2, 64
    most = -(-n // 16)
    table, pages = page_table(rng, [n] * B)  # pages of their own, as append wants them
    host = host_cache(rng, "int8", pages, Hkv, d)
    r, lens = ints(rs), ints([n] * B)
    x = _rand(rng, (n, 2, Hkv, d), "f32")
    out = torch.zeros(n, Hkv, d, device="cuda")
    for op in ("read", "attention", "append"):
        dev = DeviceCache(host, table)
        if op == "attention":
            assert dev.attention("f32", x[:, 0], r, lens, out) == 0
        else:
            assert getattr(dev, op)("f32", x[:, 0], x[:, 1], r, lens) == 0
        assert dev.err.item() == L.LLM_ERR_DEVICE, op


def test_a_call_that_failed_does_not_spoil_the_next():
    """A call into a capture that has been broken off fails; the next one, on a good stream, does not."""
    rng = np.random.default_rng(58)
    Hq, Hkv, d, rows = 4, 2, 64, 200
    table, pages = page_table(rng, [rows])
    dev = DeviceCache(host_cache(rng, "int8", pages, Hkv, d), table)
    q, out = _rand(rng, (rows, Hq, d), "f32"), torch.zeros(rows, Hq, d, device="cuda")
    rs, lens = ints([0, rows]), ints([rows])
    assert dev.attention("f32", q, rs, lens, out) == 0  # with a workspace
    torch.cuda.synchronize()
    with open("/proc/self/maps") as f:
        path = next(line.split()[-1] for line in f if "libcudart" in line)
    rt, stream, graph = ctypes.CDLL(path), ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    assert rt.cudaStreamBeginCapture(stream, 2) == 0
    assert rt.cudaStreamSynchronize(stream) != 0  # not allowed in a capture, which is void from here on
    assert dev.attention("f32", q, rs, lens, out, stream=stream) == L.LLM_ERR_CUDA
    rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
    rt.cudaGetLastError()
    x = _rand(rng, (rows, 2, Hkv, d), "f32")
    assert dev.append("f32", x[:, 0], x[:, 1], rs, lens) == 0
    assert dev.attention("f32", q, rs, lens, out) == 0
    torch.cuda.synchronize()
    assert rt.cudaStreamDestroy(stream) == 0
    assert dev.err.item() == 0
