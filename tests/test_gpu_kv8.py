"""The 8-bit K/V cache operators through the C ABI against their definitions in 64 bits (GPU required).

Codes, scales and what is read back have to be equal bit for bit: the header defines them operation by
operation.  Attention and rotation are compared within bounds that follow from their arithmetic
(tests/_kv8.py, and below)."""
import numpy as np
import pytest
import torch

from oracle import kv8
from quantized_decode_gb300 import _lib as L

from ._kv8 import DTYPES, DeviceCache, as_f32, attention_bounds, host_cache, ints, new_workspace, page_table, starts

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128), (3, 3, 64), (8, 1, 128)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    L.load()


def _rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DTYPES[dtype][0]).cuda()


# ---------------------------------------------------------------- q/k norm and rotation


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("n,norm", [(1, True), (1, False), (5, True), (333, True), (2500, False)])
def test_qk_norm_rope(dtype, Hq, Hkv, d, n, norm):
    rng = np.random.default_rng(n + Hq)
    qkv = _rand(rng, (n, (Hq + 2 * Hkv) * d), dtype, 3.0)
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    pos[0] = (1 << 20) - 1
    if n > 2:
        pos[1], pos[2] = 0, -7
    gains = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]
    qo = torch.empty(n, Hq, d, dtype=qkv.dtype, device="cuda")
    ko = torch.empty(n, Hkv, d, dtype=qkv.dtype, device="cuda")
    p = ints(pos)
    at, size = qkv.data_ptr(), qkv.element_size()
    rc = L.load().llm_op_qk_norm_rope(DTYPES[dtype][1], at, qkv.shape[1], at + Hq * d * size, qkv.shape[1],
                                      gains[0].data_ptr() if norm else None, gains[1].data_ptr() if norm else None, 1e-6, 1e6,
                                      p.data_ptr(), n, Hq, Hkv, d, qo.data_ptr(), ko.data_ptr(), None)
    assert rc == 0
    x = as_f32(qkv).reshape(n, -1, d)
    # products and sums in fp32 of values up to the pair's size: the norm's sum of d squares (d 2^-24 at worst, halved by the
    # root), its root and three products, sine and cosine off by 2^-22 with their angle, two products and a sum
    eps = (d / 2 + 16) * 2.0 ** -24
    step = 0 if dtype == "f32" else torch.finfo(DTYPES[dtype][0]).eps / 2
    for got, part, gain in ((qo, x[:, :Hq], gains[0]), (ko, x[:, Hq:Hq + Hkv], gains[1])):
        g = as_f32(gain) if norm else None
        ref = kv8.norm_rope(part, g, 1e-6, 1e6, pos)
        y = kv8.norm_rope(part, g, 1e-6, 1e6, np.zeros_like(pos))
        size = np.abs(y[..., :d // 2]) + np.abs(y[..., d // 2:])
        tol = eps * np.concatenate([size, size], -1) + step * np.abs(ref) + 2.0 ** -25 * (dtype == "f16")
        assert np.all(np.abs(as_f32(got) - ref) <= tol), float((np.abs(as_f32(got) - ref) / tol).max())


def test_qk_norm_rope_in_place_and_strided():
    rng = np.random.default_rng(3)
    n, Hq, Hkv, d = 37, 12, 2, 128
    wide = _rand(rng, (n, Hq + 3, d), "f32")
    q, k = wide[:, 1:1 + Hq], _rand(rng, (n, Hkv, d), "f32")
    pos = ints(np.arange(n) * 1000)
    qo, ko = torch.empty(n, Hq, d, device="cuda"), torch.empty(n, Hkv, d, device="cuda")
    lib = L.load()
    args = (None, None, 0.0, 1e4, pos.data_ptr(), n, Hq, Hkv, d)
    assert lib.llm_op_qk_norm_rope(0, q.data_ptr(), q.stride(0), k.data_ptr(), k.stride(0), *args, qo.data_ptr(), ko.data_ptr(), None) == 0
    q2, k2 = q.contiguous(), k.clone()
    assert lib.llm_op_qk_norm_rope(0, q2.data_ptr(), Hq * d, k2.data_ptr(), Hkv * d, *args, q2.data_ptr(), k2.data_ptr(), None) == 0
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


# ---------------------------------------------------------------- append and read


def _same(dev, host):
    got = dev.host()
    for x in ("ks", "vs"):
        np.testing.assert_array_equal(got[x], host[x])
    for x in ("k", "v"):
        np.testing.assert_array_equal(got[x], host[x])


STEPS = [
    [(1, 1), (1, 16), (1, 17), (0, 5)],       # (rows, kv after them): single tokens at page edges, a sequence at rest
    [(16, 16), (17, 17), (15, 31), (33, 64)],
    [(5, 20), (40, 43), (1, 48), (3, 18)],
    [(200, 203), (0, 0), (1, 160), (64, 64)],
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (28, 4, 128), (3, 3, 64)])
@pytest.mark.parametrize("step", range(len(STEPS)))
def test_append_is_exact(fmt, dtype, Hq, Hkv, d, step):
    rng = np.random.default_rng(step)
    rows, kv = zip(*STEPS[step])
    table, pages = page_table(rng, kv)
    host = host_cache(rng, fmt, pages, Hkv, d)
    dev = DeviceCache(host, table)
    n = sum(rows)
    fused = _rand(rng, (n + 2, 2, Hkv, d), dtype)  # K and V side by side, two rows behind the last sequence
    fused *= torch.rand((n + 2, 1, Hkv, 1), device="cuda").mul_(8).exp2_().to(fused.dtype)  # some grow the scale, some do not
    k, v = fused[:, 0], fused[:, 1]
    assert dev.append(dtype, k, v, ints(starts(rows)), ints(kv)) == 0
    kv8.append(host, table, starts(rows), kv, as_f32(k), as_f32(v))
    _same(dev, host)
    assert dev.err.item() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_token_by_token(fmt):
    """A page that grows token by token: requantised as often as a larger one comes."""
    rng = np.random.default_rng(9)
    Hkv, d, steps = 2, 128, 40
    table, pages = page_table(rng, [steps, steps])
    host = host_cache(rng, fmt, pages, Hkv, d)
    dev = DeviceCache(host, table)
    for i in range(steps):
        x = _rand(rng, (2, 2, Hkv, d), "f32", float(rng.choice([0.1, 1.0, 4.0])))
        kv = [i + 1, i + 1]
        assert dev.append("f32", x[:, 0], x[:, 1], ints([0, 1, 2]), ints(kv)) == 0
        kv8.append(host, table, [0, 1, 2], kv, as_f32(x[:, 0]), as_f32(x[:, 1]))
    _same(dev, host)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_values_at_the_edges(fmt):
    """Zeros, denormals, the largest numbers, half steps; a NaN or an infinity poisons its block alone."""
    rng = np.random.default_rng(10)
    Hkv, d = 8, 64
    table, pages = page_table(rng, [40])
    host = host_cache(rng, fmt, pages, Hkv, d)
    dev = DeviceCache(host, table)
    x = rng.standard_normal((20, 2, Hkv, d)).astype(np.float32)
    x[:, :, 0] = 0.0
    x[:, :, 1] *= np.float32(1e-41)
    x[:, :, 2] *= np.float32(5e37)
    x[:, :, 3] = np.where(np.arange(d) % 2 == 0, 127.0, np.arange(d) - 31.5).astype(np.float32)
    x[3, 0, 4, 7] = np.nan
    x[15, 1, 5, 0] = np.inf
    x[0, 0, 6, :] = np.float32(1e-45)
    x[1:, 0, 6, :] = 0.0
    x[:, 1, 6, :] = np.where(np.arange(d) == 0, 448.0, 2.0 ** -10 * (np.arange(d) % 7)).astype(np.float32)
    t = torch.from_numpy(x).cuda()
    for a, z, kv in ((0, 10, 10), (10, 20, 20)):
        y = t[a:z]
        assert dev.append("f32", y[:, 0], y[:, 1], ints([0, z - a]), ints([kv])) == 0
        kv8.append(host, table, [0, z - a], [kv], x[a:z, 0], x[a:z, 1])
    _same(dev, host)
    assert np.isnan(host["ks"][table[0, 0], 4]) and not np.isnan(host["ks"][table[0, 1], 4])
    assert np.isnan(host["vs"][table[0, 0], 5])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (28, 4, 128)])
def test_read_is_exact(fmt, dtype, Hq, Hkv, d):
    rng = np.random.default_rng(11)
    rows, kv = (1, 0, 33, 7, 100), (1, 5, 33, 20, 1000)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, fmt, pages, Hkv, d)
    dev = DeviceCache(host, table)
    n = sum(rows)
    out = torch.full((n + 3, 2, Hkv, d), 77.0, dtype=DTYPES[dtype][0], device="cuda")
    assert dev.read(dtype, out[:, 0], out[:, 1], ints(starts(rows)), ints(kv)) == 0
    for got, ref in zip((out[:, 0], out[:, 1]), kv8.read(host, table, starts(rows), kv, n)):
        assert torch.equal(got[:n].cpu(), torch.from_numpy(ref).to(DTYPES[dtype][0]))
    assert torch.all(out[n:] == 77.0)  # rows behind the last sequence
    assert dev.err.item() == 0


# ---------------------------------------------------------------- attention


def _attend(dev, host, table, dtype, q, rows, kv, check_err=0, extra=0, stream=None):
    n, Hq, d = q.shape
    out = torch.full((n, Hq, d), 55.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n, Hq), 55.0, device="cuda")
    assert dev.attention(dtype, q, ints(starts(rows)), ints(kv), out, lse, stream=stream) == 0
    torch.cuda.synchronize()
    assert dev.err.item() == check_err
    live = n - extra
    ref = kv8.attention(host, table, starts(rows), kv, as_f32(q[:live]))
    tol, ltol = attention_bounds(dtype, *ref, max(max(kv), 1))
    got, glse = as_f32(out)[:live], lse.cpu().numpy()[:live]
    empty = np.isneginf(ref[1])
    assert np.all(np.isneginf(glse[empty])) and np.all(got[empty] == 0)
    bad = np.abs(got - ref[0]) / tol
    assert np.all(bad <= 1), (float(bad.max()), np.argwhere(bad > 1)[:4])
    assert np.all(np.abs(glse[~empty] - ref[1][~empty]) <= ltol[~empty])
    assert torch.all(out[live:] == 55.0) and torch.all(lse[live:] == 55.0)
    return out, lse


CALLS = {
    "one token": ((1,), (1,)),
    "page edges": ((1, 1, 1, 1, 1), (15, 16, 17, 31, 33)),
    "one long": ((1,), (4097,)),
    "ragged": ((1, 1, 1, 0, 1, 1, 1, 1), (3000, 1, 700, 9, 16, 257, 64, 1025)),
    "drafts": ((4, 4, 2, 0, 1), (900, 4, 33, 100, 17)),
    "drafts, wide": ((9, 5, 12), (100, 300, 12)),
    "prompts": ((70, 33, 1), (70, 300, 129)),
}


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("call", list(CALLS))
def test_attention(fmt, dtype, Hq, Hkv, d, call):
    rows, kv = CALLS[call]
    rng = np.random.default_rng(len(call) + Hq)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, fmt, pages, Hkv, d)
    for b, n in enumerate(kv):  # the slots behind the last token hold anything
        if n % 16:
            host["k"][table[b, n // 16], :, n % 16:] = 0x7F
            host["v"][table[b, n // 16], :, n % 16:] = 0xFF
    dev = DeviceCache(host, table)
    q = _rand(rng, (sum(rows) + 2, Hq, d), dtype, 2.0)
    _attend(dev, host, table, dtype, q, rows, kv, extra=2)
    _attend(dev, host, table, dtype, q, rows, kv, extra=2)  # the workspace is ready for the next call


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_long_and_uneven(dtype):
    rng = np.random.default_rng(21)
    rows, kv = (1, 1, 1), (50000, 16, 3333)
    Hq, Hkv, d = 14, 2, 128
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "int8", pages, Hkv, d)
    q = _rand(rng, (3, Hq, d), dtype, 2.0)
    _attend(DeviceCache(host, table), host, table, dtype, q, rows, kv)


def test_attention_many_sequences():
    """More sequences than a warp looks at in one step, more segments than CTAs."""
    rng = np.random.default_rng(22)
    n = 150
    kv = tuple(int(x) for x in rng.integers(1, 400, n))
    rows = tuple(int(x) for x in rng.integers(0, 2, n))
    Hq, Hkv, d = 8, 4, 64
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "e4m3", pages, Hkv, d)
    q = _rand(rng, (sum(rows), Hq, d), "f32", 2.0)
    _attend(DeviceCache(host, table), host, table, "f32", q, rows, kv)


PROMPTS = {  # by rows and lengths: several blocks of 128 tokens, tiles and pairs of tiles that end anywhere
    "deep": ((200,), (1500,)),
    "from the start": ((513, 0, 300), (513, 40, 300)),
    "behind others": ((65, 1, 129, 64), (1024, 700, 129, 2000)),
}


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (7, 1, 128), (8, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("call", list(PROMPTS))
def test_attention_prompts_of_many_blocks(fmt, dtype, Hq, Hkv, d, call):
    rows, kv = PROMPTS[call]
    rng = np.random.default_rng(len(call) + Hq + d)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, fmt, pages, Hkv, d)
    q = _rand(rng, (sum(rows) + 1, Hq, d), dtype, 2.0)
    dev = DeviceCache(host, table)
    first = _attend(dev, host, table, dtype, q, rows, kv, extra=1)
    for _ in range(3):  # the result does not depend on the run
        again = _attend(dev, host, table, dtype, q, rows, kv, extra=1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("fmt,dtype", [("int8", "f32"), ("e4m3", "f32"), ("int8", "bf16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("rows,kv", [((1, 1), (700, 1300)), ((4, 3), (700, 90)), ((150, 40), (700, 300))])
@pytest.mark.parametrize("spread", [10, 40])
def test_attention_scales_far_apart(fmt, dtype, rows, kv, spread):
    """V scales of neighbouring pages up to 2^(2 spread) apart, zeros among them: rows see what is theirs, whatever pages behind
    them hold."""
    rng = np.random.default_rng(28 + spread)
    Hq, Hkv, d = 6, 2, 128
    table, pages = page_table(rng, kv)
    host = host_cache(rng, fmt, pages, Hkv, d)
    host["vs"] *= np.float32(2.0) ** rng.integers(-spread, spread + 1, host["vs"].shape).astype(np.float32)
    host["vs"][rng.random(host["vs"].shape) < 0.1] = 0
    host["ks"][rng.random(host["ks"].shape) < 0.1] = 0
    q = _rand(rng, (sum(rows), Hq, d), dtype, 2.0)
    _attend(DeviceCache(host, table), host, table, dtype, q, rows, kv)


@pytest.mark.parametrize("rows", [1, 4, 300])
def test_attention_scales_at_the_ends_of_fp32(rows):
    """V scales that fall by 2^240 along a sequence: the largest decide, nothing overflows on the way."""
    rng = np.random.default_rng(29)
    Hq, Hkv, d, kv = 4, 2, 64, 1600
    table, pages = page_table(rng, [kv])
    host = host_cache(rng, "int8", pages, Hkv, d)
    for order in (1, -1):
        host["vs"][table[0]] = (np.float32(2.0) ** np.linspace(110, -130, 100)[::order].astype(np.float32))[:, None]
        q = _rand(rng, (rows, Hq, d), "f32", 0.1)  # near even weights: every page counts by its scale
        _attend(DeviceCache(host, table), host, table, "f32", q, (rows,), (kv,))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("kv", [1, 40, 129, 1000, 5000])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (7, 1, 128)])
def test_few_rows_in_a_long_table(dtype, kv, Hq, Hkv, d):
    """Prompts too small for all SMs share their keys among CTAs by the table's length: those without keys, rows before
    the first token and pairs of tiles that are not full change nothing."""
    rng = np.random.default_rng(38 + kv)
    rows = 90
    table, pages = page_table(rng, [kv], capacity=[5008])
    host = host_cache(rng, "e4m3", pages, Hkv, d)
    q = _rand(rng, (rows + 1, Hq, d), dtype, 2.0)
    dev = DeviceCache(host, table)
    first = _attend(dev, host, table, dtype, q, (rows,), (kv,), extra=1)
    for _ in range(3):
        again = _attend(dev, host, table, dtype, q, (rows,), (kv,), extra=1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_prompt_with_a_page_that_is_none():
    rng = np.random.default_rng(30)
    Hq, Hkv, d, rows, kv = 4, 2, 64, 200, 300
    table, pages = page_table(rng, [kv])
    host = host_cache(rng, "e4m3", pages, Hkv, d)
    q = _rand(rng, (rows, Hq, d), "f32")
    for bad in (-1, pages, 1 << 30):
        t = table.copy()
        t[0, 3] = bad  # tokens 48 .. 63, which every row sees
        dev = DeviceCache(host, t)
        out = torch.zeros(rows, Hq, d, device="cuda")
        assert dev.attention("f32", q, ints([0, rows]), ints([kv]), out) == 0
        assert dev.err.item() == L.LLM_ERR_DEVICE
        # the same tokens in a sequence without that page
        short = DeviceCache(host, np.delete(table, 3, axis=1))
        want = torch.zeros(rows, Hq, d, device="cuda")
        assert short.attention("f32", q, ints([0, rows]), ints([kv - 16]), want) == 0
        assert short.err.item() == 0
        # both within 2 (36 2^-23 A + 2^-21) + 800 2^-23 of sums w|v| below 6, with A = sum|q k| / 8 below 300
        assert float((out - want).abs().max()) < 2 * 6 * (2 * (300 * 36 * 2.0 ** -23 + 2.0 ** -21) + 800 * 2.0 ** -23)


def test_many_sequences_in_one_call():
    """Append, read and prompt attention with more sequences than a warp looks at in one step, some of them empty."""
    rng = np.random.default_rng(35)
    n, Hq, Hkv, d = 150, 6, 3, 64
    rows = rng.integers(0, 60, n)
    rows[rng.random(n) < 0.2] = 0
    kv = rows + rng.integers(0, 40, n)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "int8", pages, Hkv, d)
    dev = DeviceCache(host, table)
    k, v = (_rand(rng, (int(rows.sum()), Hkv, d), "bf16") for _ in range(2))
    rs, lens = ints(starts(rows)), ints(kv)
    assert dev.append("bf16", k, v, rs, lens) == 0
    kv8.append(host, table, starts(rows), kv, as_f32(k), as_f32(v))
    got = dev.host()
    for x in ("k", "v", "ks", "vs"):
        np.testing.assert_array_equal(got[x], host[x])
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    assert dev.read("bf16", ko, vo, rs, lens) == 0
    for a, ref in zip((ko, vo), kv8.read(host, table, starts(rows), kv, len(k))):
        assert torch.equal(a.cpu(), torch.from_numpy(ref).bfloat16())
    q = _rand(rng, (len(k), Hq, d), "f32", 2.0)
    _attend(dev, host, table, "f32", q, tuple(int(x) for x in rows), tuple(int(x) for x in kv))


@pytest.mark.parametrize("rows", [1, 4, 100])
def test_pages_beyond_32_bits(rows):
    """Pools of more than 4 GB, pages at their end: every offset is 64 bits wide."""
    rng = np.random.default_rng(36)
    Hq, Hkv, d, kv = 16, 8, 128, 130
    pages = 270000  # 4.4 GB of K, as much of V
    used = -(-kv // 16)
    small = host_cache(rng, "int8", used, Hkv, d)
    dev = DeviceCache(small, np.arange(used, dtype=np.int32)[None])
    k = torch.empty(pages, Hkv, 16, d, dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = (torch.zeros(pages, Hkv, device="cuda") for _ in range(2))
    for big, part in ((k, dev.k), (v, dev.v), (ks, dev.ks), (vs, dev.vs)):
        big[pages - used:] = part
    far = DeviceCache(small, np.arange(pages - used, pages, dtype=np.int32)[None])
    far.k, far.v, far.ks, far.vs, far.shape = k, v, ks, vs, tuple(k.shape)
    x = _rand(rng, (rows, 2, Hkv, d), "bf16", 3.0)
    q = _rand(rng, (rows, Hq, d), "f32")
    outs = []
    for c in (dev, far):
        rs, lens = ints([0, rows]), ints([kv])
        out, back = torch.zeros(rows, Hq, d, device="cuda"), torch.zeros_like(x)
        assert c.append("bf16", x[:, 0], x[:, 1], rs, lens) == 0
        assert c.read("bf16", back[:, 0], back[:, 1], rs, lens) == 0
        assert c.attention("f32", q, rs, lens, out) == 0
        torch.cuda.synchronize()
        assert c.err.item() == 0
        outs.append((out, back))
    assert torch.equal(far.k[pages - used:], dev.k) and torch.equal(far.vs[pages - used:], dev.vs)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_prompt_in_a_graph_on_a_side_stream():
    """A captured prompt step, replayed with other lengths than it was captured with."""
    rng = np.random.default_rng(37)
    Hq, Hkv, d, rows = 8, 2, 128, (90, 140)
    cap = (400, 300)
    table, pages = page_table(rng, cap)
    host = host_cache(rng, "e4m3", pages, Hkv, d)
    dev = DeviceCache(host, table)
    q = _rand(rng, (sum(rows), Hq, d), "bf16", 2.0)
    rs, lens = ints(starts(rows)), ints((90, 140))
    out, lse = torch.zeros(sum(rows), Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(sum(rows), Hq, device="cuda")
    space = new_workspace(dev, Hq, sum(rows))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
        assert dev.attention("bf16", q, rs, lens, out, lse, stream=torch.cuda.current_stream().cuda_stream, workspace=space) == 0
        graph.capture_end()
    for kv in ((90, 140), cap, (91, 299)):
        lens.copy_(ints(kv))
        graph.replay()
        torch.cuda.synchronize()
        ref = kv8.attention(host, table, starts(rows), kv, as_f32(q))
        tol, ltol = attention_bounds("bf16", *ref, max(kv))
        assert np.all(np.abs(as_f32(out) - ref[0]) <= tol) and np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_attention_rows_that_see_nothing(rows):
    rng = np.random.default_rng(23)
    Hq, Hkv, d = 12, 2, 128
    table, pages = page_table(rng, [16, 16, 32])
    host = host_cache(rng, "int8", pages, Hkv, d)
    q = _rand(rng, (3 * rows, Hq, d), "f32", 2.0)
    _attend(DeviceCache(host, table), host, table, "f32", q, (rows,) * 3, (0, min(2, rows), 20))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_wide_scores_and_strided_q(dtype):
    """Scores of hundreds, rows of very different size, q inside fused rows."""
    rng = np.random.default_rng(24)
    Hq, Hkv, d, kv, rows = 12, 2, 128, (333, 70), (2, 3)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "int8", pages, Hkv, d)
    fused = _rand(rng, (5, Hq + 4, d), dtype, 1.0)
    fused *= torch.tensor([1e-3, 1.0, 30.0, 200.0, 0.0], device="cuda").to(fused.dtype)[:, None, None]
    _attend(DeviceCache(host, table), host, table, dtype, fused[:, 2:2 + Hq], rows, kv)


def test_attention_nan_blocks_stay_where_they_are():
    """A NaN scale makes NaN of the rows and heads that see its block, and of no other."""
    rng = np.random.default_rng(25)
    Hq, Hkv, d, kv, rows = 4, 2, 64, (40, 40), (30, 1)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "e4m3", pages, Hkv, d)
    clean = DeviceCache(host, table)
    host["vs"][table[0, 1], 1] = np.nan  # tokens 16 .. 31 of sequence 0, V of head 1
    host["ks"][table[0, 2], 0] = np.nan  # tokens 32 .. of sequence 0, K of head 0
    dev = DeviceCache(host, table)
    q = _rand(rng, (31, Hq, d), "f32")
    outs = []
    for c in (clean, dev):
        out = torch.zeros(31, Hq, d, device="cuda")
        assert c.attention("f32", q, ints([0, 30, 31]), ints(kv), out) == 0
        outs.append(out.cpu())
    a, b = outs
    hit = torch.zeros(31, Hq, dtype=torch.bool)
    hit[6:30, 2:] = True   # rows at positions 16 .. see V of head 1's block
    hit[22:30, :2] = True  # rows at positions 32 .. see K of head 0's block
    assert torch.all(torch.isnan(b[hit])) and torch.equal(a[~hit], b[~hit])


def test_numbers_out_of_range_are_reported_and_left_out():
    """Bad pages, lengths and row starts: nothing out of range is touched, err says so, the rest is right."""
    rng = np.random.default_rng(26)
    Hq, Hkv, d, rows, kv = 4, 2, 64, (1, 1, 1), (40, 40, 40)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "int8", pages, Hkv, d)
    q = _rand(rng, (3, Hq, d), "f32")
    for bad in (-1, pages, 1 << 30):  # a page that is none: its tokens are left out
        t = table.copy()
        t[1, 1] = bad
        dev = DeviceCache(host, t)
        out = torch.zeros(3, Hq, d, device="cuda")
        assert dev.attention("f32", q, ints(starts(rows)), ints(kv), out) == 0
        assert dev.err.item() == L.LLM_ERR_DEVICE
        other = {**host, "k": host["k"].copy(), "v": host["v"].copy(), "ks": host["ks"].copy(), "vs": host["vs"].copy()}
        ref = kv8.attention(other, table, starts(rows), kv, as_f32(q))[0]
        got = as_f32(out)
        np.testing.assert_allclose(got[[0, 2]], ref[[0, 2]], atol=1e-4)
        keep = np.r_[0:16, 32:40]
        for h in range(Hq):
            g = h // 2
            K = (kv8.decode(host["k"][table[1], g], "int8") * host["ks"][table[1], g][:, None, None]).reshape(-1, d)[keep]
            V = (kv8.decode(host["v"][table[1], g], "int8") * host["vs"][table[1], g][:, None, None]).reshape(-1, d)[keep]
            w = np.exp(K @ as_f32(q)[1, h] / 8)
            np.testing.assert_allclose(got[1, h], w @ V / w.sum(), atol=1e-4)
        x = _rand(rng, (3, 2, Hkv, d), "f32")
        dev.err.zero_()
        t2 = table.copy()
        t2[1, 2] = bad
        dev = DeviceCache(host, t2)
        assert dev.append("f32", x[:, 0], x[:, 1], ints(starts(rows)), ints(kv)) == 0
        assert dev.err.item() == L.LLM_ERR_DEVICE
        changed = (dev.k.cpu().numpy() != host["k"]).any((1, 2, 3))
        assert set(np.flatnonzero(changed)) <= {table[0, 2], table[2, 2]}
        dev.err.zero_()
        out = torch.full((3, 2, Hkv, d), 5.0, device="cuda")
        assert dev.read("f32", out[:, 0], out[:, 1], ints(starts(rows)), ints(kv)) == 0
        assert dev.err.item() == L.LLM_ERR_DEVICE and torch.all(out[1] == 5.0) and not torch.any(out[[0, 2]] == 5.0)
    for bad_kv in (-1, 49, 1 << 30, -(1 << 31)):  # the table holds 48 tokens
        dev = DeviceCache(host, table)
        lens = (40, bad_kv, 40)
        out, lse = torch.full((3, Hq, d), 5.0, device="cuda"), torch.zeros(3, Hq, device="cuda")
        assert dev.attention("f32", q, ints(starts(rows)), ints(lens), out, lse) == 0
        assert dev.err.item() == L.LLM_ERR_DEVICE
        assert torch.all(out[1] == 0) and torch.all(lse[1] == -float("inf")) and torch.all(out[[0, 2]] != 0)
        for call in (dev.append, dev.read):
            dev.err.zero_()
            x = torch.full((3, 2, Hkv, d), 5.0, device="cuda")
            assert call("f32", x[:, 0], x[:, 1], ints(starts(rows)), ints(lens)) == 0
            assert dev.err.item() == L.LLM_ERR_DEVICE and torch.all(x[1] == 5.0)
    for rs in ([0, 1, 9, 9], [0, 2, 1, 3], [-4, 1, 2, 3], [0, 1 << 30, 1 << 30, 1 << 30]):
        dev = DeviceCache(host, table)
        out = torch.full((3, Hq, d), 5.0, device="cuda")
        assert dev.attention("f32", q, ints(rs), ints(kv), out) == 0
        assert dev.err.item() == L.LLM_ERR_DEVICE
        for call in (dev.append, dev.read):
            dev.err.zero_()
            x = torch.full((3, 2, Hkv, d), 5.0, device="cuda")
            assert call("f32", x[:, 0], x[:, 1], ints(rs), ints(kv)) == 0
            torch.cuda.synchronize()
            assert dev.err.item() == L.LLM_ERR_DEVICE
    dev = DeviceCache(host, table)  # more rows than tokens: refused where rows are written or read
    x = torch.full((9, 2, Hkv, d), 5.0, device="cuda")
    assert dev.append("f32", x[:, 0], x[:, 1], ints([0, 3, 6, 9]), ints([2, 40, 40])) == 0
    assert dev.err.item() == L.LLM_ERR_DEVICE


# ---------------------------------------------------------------- streams, graphs, the whole chain


def test_results_do_not_depend_on_the_run():
    rng = np.random.default_rng(31)
    Hq, Hkv, d, rows, kv = 28, 4, 128, (1, 1, 4), (5000, 77, 1200)
    table, pages = page_table(rng, kv)
    dev = DeviceCache(host_cache(rng, "e4m3", pages, Hkv, d), table)
    q = _rand(rng, (6, Hq, d), "f32")
    first = None
    for _ in range(20):
        out, lse = torch.zeros(6, Hq, d, device="cuda"), torch.zeros(6, Hq, device="cuda")
        assert dev.attention("f32", q, ints(starts(rows)), ints(kv), out, lse) == 0
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_two_streams_with_their_own_workspaces():
    rng = np.random.default_rng(32)
    Hq, Hkv, d, kv = 28, 4, 128, (20000,)
    table, pages = page_table(rng, kv)
    dev = DeviceCache(host_cache(rng, "int8", pages, Hkv, d), table)
    rs, lens = ints([0, 1]), ints(kv)
    qs = [_rand(rng, (1, Hq, d), "f32") for _ in range(2)]
    want = [torch.zeros(1, Hq, d, device="cuda") for _ in range(2)]
    for q, w in zip(qs, want):
        assert dev.attention("f32", q, rs, lens, w) == 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [new_workspace(dev, Hq, 1) for _ in range(2)]
    outs = [[torch.zeros(1, Hq, d, device="cuda") for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for j in range(2):
            assert dev.attention("f32", qs[j], rs, lens, outs[j][i], stream=streams[j].cuda_stream, workspace=spaces[j]) == 0
    torch.cuda.synchronize()
    for j in range(2):
        for o in outs[j]:
            assert torch.equal(o, want[j])


@pytest.mark.parametrize("fmt,dtype", [("int8", "f32"), ("e4m3", "bf16")])
def test_decode_steps_in_a_graph(fmt, dtype):
    """Rotation, append and attention of a layer as one captured graph, replayed as two sequences grow, against the
    definitions run on the same rows."""
    rng = np.random.default_rng(33)
    Hq, Hkv, d, steps = 12, 2, 128, 21
    lens = np.array([30, 5], np.int32)
    table, pages = page_table(rng, lens, capacity=lens + steps)
    host = host_cache(rng, fmt, pages, Hkv, d)
    dev = DeviceCache(host, table)
    tdt, tid = DTYPES[dtype]
    qkv = torch.zeros(2, (Hq + 2 * Hkv) * d, dtype=tdt, device="cuda")
    gains = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]
    pos, kv, rs = ints(lens - 1), ints(lens), ints([0, 1, 2])
    qo = torch.zeros(2, Hq, d, dtype=tdt, device="cuda")
    ko = torch.zeros(2, Hkv, d, dtype=tdt, device="cuda")
    out, lse = torch.zeros(2, Hq, d, dtype=tdt, device="cuda"), torch.zeros(2, Hq, device="cuda")
    v = qkv[:, (Hq + Hkv) * d:].view(2, Hkv, d)
    space = new_workspace(dev, Hq, 2)
    lib = L.load()

    def step(stream):
        at, size = qkv.data_ptr(), qkv.element_size()
        assert lib.llm_op_qk_norm_rope(tid, at, qkv.shape[1], at + Hq * d * size, qkv.shape[1], gains[0].data_ptr(),
                                       gains[1].data_ptr(), 1e-6, 1e6, pos.data_ptr(), 2, Hq, Hkv, d, qo.data_ptr(),
                                       ko.data_ptr(), stream) == 0
        assert dev.append(dtype, ko, v, rs, kv, stream=stream) == 0
        assert dev.attention(dtype, qo, rs, kv, out, lse, stream=stream, workspace=space) == 0

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
        step(torch.cuda.current_stream().cuda_stream)
        graph.capture_end()
    for i in range(steps):
        x = _rand(rng, tuple(qkv.shape), dtype)
        qkv.copy_(x)
        pos.copy_(ints(lens + i))
        kv.copy_(ints(lens + i + 1))
        graph.replay()
        torch.cuda.synchronize()
        xs = as_f32(x).reshape(2, -1, d)
        # the rotation within its own bounds (tested above); what the cache holds follows from its rows exactly
        kref = kv8.norm_rope(xs[:, Hq:Hq + Hkv], as_f32(gains[1]), 1e-6, 1e6, lens + i)
        np.testing.assert_allclose(as_f32(ko), kref, rtol=0.01, atol=0.02)
        kv8.append(host, table, [0, 1, 2], lens + i + 1, as_f32(ko), as_f32(v))
        _same(dev, host)
        ref = kv8.attention(host, table, [0, 1, 2], lens + i + 1, as_f32(qo))
        tol, ltol = attention_bounds(dtype, *ref, int(lens.max()) + i + 1)
        assert np.all(np.abs(as_f32(out) - ref[0]) <= tol)
        assert np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)
    assert dev.err.item() == 0


def test_prompt_then_steps_against_the_bf16_attention():
    """A prompt and some decode steps through the 8-bit cache stay within quantisation of the engine's attention over the
    same K and V in bf16: K off by half a step of its block's scale moves a score by at most sum|q| s / (2 sqrt(d)), V by s / 2."""
    rng = np.random.default_rng(34)
    Hq, Hkv, d, prompt, total = 28, 4, 128, 90, 97
    table, pages = page_table(rng, [total])
    host = host_cache(rng, "int8", pages, Hkv, d)
    dev = DeviceCache(host, table)
    k, v = (_rand(rng, (total, Hkv, d), "bf16") for _ in range(2))
    q = _rand(rng, (total, Hq, d), "f32")
    outs = torch.zeros(total, Hq, d, device="cuda")
    assert dev.append("bf16", k[:prompt], v[:prompt], ints([0, prompt]), ints([prompt])) == 0
    assert dev.attention("f32", q[:prompt], ints([0, prompt]), ints([prompt]), outs[:prompt]) == 0
    for i in range(prompt, total):
        assert dev.append("bf16", k[i:i + 1], v[i:i + 1], ints([0, 1]), ints([i + 1])) == 0
        assert dev.attention("f32", q[i:i + 1], ints([0, 1]), ints([i + 1]), outs[i:i + 1]) == 0
    kp = torch.zeros(pages, Hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    for i in range(total):
        kp[table[0, i // 16], :, i % 16] = k[i]
        vp[table[0, i // 16], :, i % 16] = v[i]
    scale = dev.host()
    for i in (0, 5, prompt - 1, prompt, total - 1):
        ref = torch.zeros(Hq, d, device="cuda")
        assert L.load().llm_op_attention(q[i].data_ptr(), kp.data_ptr(), vp.data_ptr(), dev.table.data_ptr(), pages, i + 1, Hq,
                                         Hkv, d, 0, ref.data_ptr(), None) == 0
        for h in range(Hq):
            ks, vs = (scale[x][table[0, :i // 16 + 1], h // (Hq // Hkv)].max() for x in ("ks", "vs"))
            # two roundings at most per element here (written, and requantised once per growth: up to 7 in the steps' page)
            ds = float(q[i, h].abs().sum()) * ks * 4 / np.sqrt(d)
            most = float(v[:i + 1, h // (Hq // Hkv)].abs().max())
            tol = min(2 * most, (np.exp(2 * ds) - 1) * most) + 4 * vs
            assert float((outs[i, h] - ref[h]).abs().max()) <= tol
    # typical error: far below
    assert float((outs[total - 1] - ref).square().mean().sqrt() / ref.square().mean().sqrt()) < 0.05


# ---------------------------------------------------------------- calls at the edges of what is allowed


@pytest.mark.parametrize("rows", [(1, 2), (150, 40)])
def test_rows_before_the_first_sequence_and_strided_rows(rows):
    """row_start[0] > 0, all rows inside wider ones, no err word: rows that are nobody's stay as they are."""
    rng = np.random.default_rng(41)
    Hq, Hkv, d, first, kv = 12, 2, 64, 301, (170, 45)
    n = first + sum(rows) + 2
    rs = first + starts(rows)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "int8", pages, Hkv, d)
    dev = DeviceCache(host, table)
    wide = _rand(rng, (n, Hq + 2 * Hkv + 2, d), "f16", 2.0)
    q, k, v = wide[:, 1:1 + Hq], wide[:, Hq + 1:Hq + Hkv + 1], wide[:, Hq + Hkv + 1:Hq + 2 * Hkv + 1]
    lib, tid, r, lens = L.load(), DTYPES["f16"][1], ints(rs), ints(kv)
    assert lib.llm_op_kv8_append(dev.struct(), tid, k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), r.data_ptr(), lens.data_ptr(), n,
                                 None, None) == 0
    kv8.append(host, table, rs, kv, as_f32(k), as_f32(v))
    got = dev.host()
    for x in ("k", "v", "ks", "vs"):
        np.testing.assert_array_equal(got[x], host[x])
    back = torch.full((n, 2, Hkv + 1, d), 77.0, dtype=torch.float16, device="cuda")
    assert lib.llm_op_kv8_read(dev.struct(), tid, r.data_ptr(), lens.data_ptr(), n, back[:, 0].data_ptr(), back.stride(0), back[:, 1].data_ptr(),
                               back.stride(0), None, None) == 0
    for i, ref in enumerate(kv8.read(host, table, rs, kv, n)):
        assert torch.equal(back[first:first + sum(rows), i, :Hkv].cpu(), torch.from_numpy(ref[first:first + sum(rows)]).half())
    assert torch.all(back[:first] == 77) and torch.all(back[-2:] == 77) and torch.all(back[:, :, Hkv] == 77)
    out = torch.full((n, Hq, d), 55.0, dtype=torch.float16, device="cuda")
    space = new_workspace(dev, Hq, n)
    assert lib.llm_op_kv8_attention(dev.struct(), tid, q.data_ptr(), q.stride(0), r.data_ptr(), lens.data_ptr(), n, Hq, out.data_ptr(), None,
                                    space.data_ptr(), space.numel(), None, None) == 0
    ref = kv8.attention(host, table, rs, kv, as_f32(q))
    tol, _ = attention_bounds("f16", *ref, max(kv))
    mine = slice(first, first + sum(rows))
    assert np.all(np.abs(as_f32(out) - ref[0])[mine] <= tol[mine])
    assert torch.all(out[:first] == 55) and torch.all(out[-2:] == 55)


def test_the_most_sequences():
    rng = np.random.default_rng(42)
    n, Hq, Hkv, d = 4096, 2, 1, 64
    kv = rng.integers(0, 40, n)
    rows = np.minimum(kv, rng.integers(0, 3, n))
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "int8", pages, Hkv, d)
    q = _rand(rng, (int(rows.sum()), Hq, d), "f32", 2.0)
    _attend(DeviceCache(host, table), host, table, "f32", q, tuple(int(x) for x in rows), tuple(int(x) for x in kv))


@pytest.mark.parametrize("rows", [1, 70])
def test_many_heads_and_uneven_lengths(rows):
    """More heads than SMs would share evenly, one long sequence among short ones."""
    rng = np.random.default_rng(43)
    Hq, Hkv, d, kv = 40, 40, 64, (5000, 80, 300)
    table, pages = page_table(rng, kv)
    host = host_cache(rng, "e4m3", pages, Hkv, d)
    q = _rand(rng, (3 * rows, Hq, d), "bf16", 2.0)
    _attend(DeviceCache(host, table), host, table, "bf16", q, (rows,) * 3, kv)


@pytest.mark.parametrize("rows", [1, 5, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_a_row_that_is_not_finite_is_its_own_affair(rows, bad):
    rng = np.random.default_rng(44)
    Hq, Hkv, d, kv = 8, 2, 128, (700, 260)
    table, pages = page_table(rng, kv)
    dev = DeviceCache(host_cache(rng, "int8", pages, Hkv, d), table)
    q = _rand(rng, (2 * rows, Hq, d), "f32")
    outs = []
    for spoil in (False, True):
        x = q.clone()
        if spoil:
            x[rows // 2, 3, 17] = bad
        out, lse = torch.zeros_like(x), torch.zeros(2 * rows, Hq, device="cuda")
        assert dev.attention("f32", x, ints([0, rows, 2 * rows]), ints(kv), out, lse) == 0
        outs.append((out, lse))
    keep = torch.ones(2 * rows, Hq, dtype=torch.bool, device="cuda")
    keep[rows // 2, 3] = False
    assert torch.equal(outs[0][0][keep], outs[1][0][keep]) and torch.equal(outs[0][1][keep], outs[1][1][keep])
    if bad != 3e38:
        assert torch.all(torch.isnan(outs[1][0][~keep]))


def test_a_workspace_that_is_too_small_is_refused():
    rng = np.random.default_rng(45)
    table, pages = page_table(rng, [20])
    dev = DeviceCache(host_cache(rng, "int8", pages, 2, 64), table)
    q = _rand(rng, (1, 4, 64), "f32")
    out = torch.full_like(q, 9.0)
    space = new_workspace(dev, 4, 1)
    assert dev.attention("f32", q, ints([0, 1]), ints([20]), out, workspace=space[:-1]) == L.LLM_ERR_ARG
    assert torch.all(out == 9.0)
