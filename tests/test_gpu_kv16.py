"""The 16-bit K/V cache operators through the C ABI against their definitions in 64 bits (GPU required).

What is copied, chosen or counted has to be equal; rotation, attention and weights are compared within bounds that follow from
their arithmetic (tests/_kv16.py, and below)."""
import numpy as np
import pytest
import torch

from oracle import kv16
from quantized_decode_gb300 import _lib as L

from ._kv16 import DTYPES, HEADS, PAGES, Cache, as_f32, attention_bounds, ints, rand, starts, weigh_bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    L.load()


# ---------------------------------------------------------------- norm, rotation and write


def _axes(d, kind):
    h = d // 2
    if kind == "text":
        return np.zeros(h, int), 1
    if kind == "sections":
        return np.repeat([0, 1, 2], [h // 4, h * 3 // 8, h - h // 4 - h * 3 // 8]), 3
    return np.arange(h) % 8, 8


def _close(got, ref, size, dtype, pages):
    """fp32 products and sums of values up to the pair's `size`: the norm's sum of d squares (halved by the root), its root and three
    products, sine and cosine off by 2^-22 with their angle, two products and a sum; then one rounding to the pages' type."""
    eps = (ref.shape[-1] / 2 + 16) * 2.0 ** -24
    tol = eps * size + torch.finfo(PAGES[pages]).eps / 2 * np.abs(ref) + 2.0 ** -25 * (pages == "f16") + 1e-38
    bad = np.abs(got - ref) / tol
    assert np.all(bad <= 1), float(bad.max())


def _check_append(rng, dtype, pages, Hq, Hkv, d, rows, kv, axes, norm, extra=0, capacity=None):
    c = Cache(rng, pages, Hkv, d, kv, capacity=capacity)
    n = sum(rows)
    qkv = rand(rng, (n + extra, (Hq + 2 * Hkv) * d), dtype, 3.0)
    axis, n_axes = _axes(d, axes)
    pos = rng.integers(0, 1 << 20, (n_axes, n + extra)).astype(np.int32)
    pos[0, 0], pos[-1, -1] = (1 << 20) - 1, -7
    gains = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]
    out = torch.full((n + extra, Hq, d), 7.0, dtype=PAGES[pages], device="cuda")
    before = [x.clone() for x in (c.k, c.v)]
    p = ints(pos)
    assert c.rope_append(qkv, Hq, gains if norm else None, axis, n_axes, p, ints(starts(rows)), out) == 0
    assert c.err.item() == 0
    x = as_f32(qkv)[:n].reshape(n, -1, d)
    zero = np.zeros_like(pos[:, :n])
    refs = []
    for part, g in ((x[:, :Hq], gains[0]), (x[:, Hq:Hq + Hkv], gains[1])):
        gain = as_f32(g) if norm else None
        y = np.abs(kv16.rotate(part, gain, 1e-6, 1e6, axis, zero))
        size = y[..., :d // 2] + y[..., d // 2:]
        refs.append((kv16.rotate(part, gain, 1e-6, 1e6, axis, pos[:, :n]), np.concatenate([size, size], -1)))
    _close(as_f32(out)[:n], *refs[0], dtype, pages)
    assert torch.all(out[n:] == 7.0)
    at = starts(rows)
    touched = torch.zeros(c.k.shape[0], 16, dtype=torch.bool)
    for b, length in enumerate(kv):
        page, slot = (z[length - rows[b]:] for z in kv16.slots(c.table[b], length))
        touched[page, slot] = True
        mine = slice(at[b], at[b + 1])
        _close(as_f32(c.k)[page, :, slot], refs[1][0][mine], refs[1][1][mine], dtype, pages)
        v = torch.from_numpy(x[mine, Hq + Hkv:]).to(PAGES[pages])
        assert torch.equal(c.v.cpu()[page, :, slot], v)
    for now, old in zip((c.k, c.v), before):
        same = (now == old).all(-1).all(1).cpu()
        assert bool(same[~touched].all())  # slots of no row


@pytest.mark.parametrize("dtype,pages", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("axes,norm", [("sections", True), ("each", False)])
def test_rope_append(dtype, pages, Hq, Hkv, d, axes, norm):
    rng = np.random.default_rng(Hq + d)
    _check_append(rng, dtype, pages, Hq, Hkv, d, (1, 0, 33, 16, 5), (1, 7, 40, 16, 1000), axes, norm, extra=2)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,kv", [((1,), (1,)), ((1,) * 70, tuple(range(1, 71))), ((900, 1, 700), (900, 17, 3000)), ((3,) * 33, (48,) * 33)])
def test_rope_append_many(dtype, rows, kv):
    _check_append(np.random.default_rng(len(rows)), dtype, "bf16", 28, 4, 128, rows, kv, "text", True)


def test_rope_append_like_the_one_axis_operator():
    """All axes alike: q is what llm_op_qk_norm_rope gives for the same rows."""
    rng = np.random.default_rng(5)
    n, Hq, Hkv, d = 50, 12, 2, 128
    c = Cache(rng, "bf16", Hkv, d, [n])
    qkv = rand(rng, (n, (Hq + 2 * Hkv) * d), "bf16", 3.0)
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    out, q1 = (torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k1 = torch.empty(n, Hkv, d, dtype=torch.bfloat16, device="cuda")
    three, one = ints(np.stack([pos] * 3)), ints(pos)
    assert c.rope_append(qkv, Hq, None, _axes(d, "sections")[0], 3, three, ints([0, n]), out) == 0
    at, w = qkv.data_ptr(), qkv.shape[1]
    assert L.load().llm_op_qk_norm_rope(2, at, w, at + Hq * d * 2, w, None, None, 1e-6, 1e6, one.data_ptr(), n, Hq, Hkv, d, q1.data_ptr(),
                                        k1.data_ptr(), None) == 0
    page, slot = kv16.slots(c.table[0], n)
    assert torch.equal(out, q1) and torch.equal(c.k.cpu()[page, :, slot], k1.cpu())


def test_rope_append_copies_v_as_it_is():
    """Infinities, NaN and the largest numbers of V; a NaN of one head stays there."""
    rng = np.random.default_rng(6)
    n, Hq, Hkv, d = 20, 4, 2, 64
    c = Cache(rng, "bf16", Hkv, d, [n])
    qkv = rand(rng, (n, Hq + 2 * Hkv, d), "f32")
    qkv[3, Hq + Hkv, 5], qkv[4, Hq + Hkv, 6], qkv[5, Hq + Hkv, 7], qkv[6, Hq + Hkv, 8] = np.inf, -np.inf, np.nan, 3e38
    qkv[7, 1, 3] = np.nan
    out = torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda")
    gains = [torch.ones(d, dtype=torch.bfloat16, device="cuda")] * 2
    assert c.rope_append(qkv.view(n, -1), Hq, gains, np.zeros(32, int), 1, ints(np.arange(n)[None]), ints([0, n]), out) == 0
    page, slot = kv16.slots(c.table[0], n)
    got, ref = c.v.cpu()[page, :, slot], qkv[:, Hq + Hkv:].bfloat16().cpu()
    assert torch.equal(got.view(torch.int16)[~ref.isnan()], ref.view(torch.int16)[~ref.isnan()]) and bool(got[ref.isnan()].isnan().all())
    bad = out.isnan().any(-1)
    assert bool(bad[7, 1]) and bad.sum() == 1 and not bool(c.k.cpu()[page, :, slot].isnan().any())


# ---------------------------------------------------------------- attention


def _attend(c, q, rows, kv, extra=0, check_err=0, **kw):
    n, Hq, d = q.shape
    out, lse = torch.full((n, Hq, d), 55.0, dtype=q.dtype, device="cuda"), torch.full((n, Hq), 55.0, device="cuda")
    rs = ints(starts(rows))
    assert c.attention(q, rs, out, lse, **kw) == 0
    torch.cuda.synchronize()
    assert c.err.item() == check_err
    return out, lse


def _check_attention(c, q, rows, kv, extra=0):
    out, lse = _attend(c, q, rows, kv, extra)
    live = q.shape[0] - extra
    ref = kv16.attention(*c.host(), c.table, starts(rows), kv, as_f32(q[:live]), c.prefix)
    tol, ltol = attention_bounds(c.dtype, *ref, max(kv) + max(c.prefix[1] if c.prefix else [0]))
    got, glse = as_f32(out)[:live], lse.cpu().numpy()[:live]
    empty = np.isneginf(ref[1])
    assert np.all(np.isneginf(glse[empty])) and np.all(got[empty] == 0)
    bad = np.abs(got - ref[0]) / tol
    assert np.all(bad <= 1), (float(np.nanmax(bad)), np.argwhere(~(bad <= 1))[:4])
    bad = np.abs(glse[~empty] - ref[1][~empty]) / ltol[~empty]
    assert np.all(bad <= 1), float(bad.max())
    assert torch.all(out[live:] == 55.0) and torch.all(lse[live:] == 55.0)
    return out, lse


# (rows, kv) of each sequence; (prefix lengths, seq_start)
SHAPES = {
    "one token": ([(1, 1)], None),
    "no token of its own behind a prefix": ([(1, 0), (1, 1)], ([5], [0, 2])),
    "page edges": ([(1, 15), (1, 16), (1, 17), (0, 9), (1, 31), (1, 33)], None),
    "steps behind one prefix": ([(1, 1), (1, 30), (1, 100), (1, 64)], ([200], [0, 4])),
    "prefix of one token": ([(1, 3), (1, 20)], ([1], [0, 2])),
    "empty prefix": ([(1, 3), (2, 20)], ([0], [0, 2])),
    "prefix at block edges": ([(1, 3), (2, 20), (1, 7)], ([128, 127, 129], [0, 1, 2, 3])),
    "drafts": ([(5, 5), (4, 100), (3, 16), (5, 700)], ([300], [0, 4])),
    "groups and loners": ([(1, 20)] * 9, ([100, 0, 257], [1, 4, 4, 8])),
    "prompts": ([(130, 130), (1, 1), (64, 200), (300, 333)], ([140], [0, 4])),
    "prompts alone": ([(257, 257), (129, 640)], None),
    "more rows than tokens": ([(5, 2), (1, 0), (3, 3)], None),
    "more rows than tokens behind a prefix": ([(5, 2), (1, 0), (3, 3)], ([40], [0, 3])),
    "long prefix": ([(1, 40)] * 5, ([3000], [0, 5])),
    "long own": ([(1, 5000), (2, 700)], ([33], [0, 2])),
    "many sequences": ([(1, 1 + 7 * (i % 13)) for i in range(150)], ([500, 300], [0, 100, 150])),
}


@pytest.mark.parametrize("dtype", list(PAGES))
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_attention(dtype, Hq, Hkv, d, shape):
    seqs, prefix = SHAPES[shape]
    if shape in ("prompts", "prompts alone", "many sequences") and Hq > 12:
        seqs = seqs[:100]
        prefix = prefix and (prefix[0], [min(x, len(seqs)) for x in prefix[1]])
    rng = np.random.default_rng(len(shape) + Hq)
    rows, kv = zip(*seqs)
    c = Cache(rng, dtype, Hkv, d, kv, prefix)
    q = rand(rng, (sum(rows) + 2, Hq, d), dtype, 2.0)
    _check_attention(c, q, rows, kv, extra=2)


@pytest.mark.parametrize("dtype", list(PAGES))
def test_attention_does_not_see_what_lies_behind(dtype):
    """NaN and infinities in slots behind the last token, behind a prefix and in pages of nobody."""
    rng = np.random.default_rng(3)
    for rows, kv, prefix in (((1, 1, 3), (5, 17, 40), ([21], [0, 3])), ((150, 1), (150, 3), ([130], [0, 2])), ((70, 200), (75, 210), None)):
        c = Cache(rng, dtype, 2, 128, kv, prefix)
        seen = torch.zeros(c.pages, 16, dtype=torch.bool)
        for table, lens in ((c.table, kv), *([c.prefix[:2]] if prefix else [])):
            for b, n in enumerate(lens):
                seen[kv16.slots(table[b], n)] = True
        hide = ~seen.cuda()
        q = rand(rng, (sum(rows), 12, 128), dtype, 2.0)
        out, lse = _attend(c, q, rows, kv)
        for x, bad in ((c.k, float("nan")), (c.v, float("inf")), (c.v, float("nan")), (c.k, float("-inf"))):
            x.permute(0, 2, 1, 3)[hide] = bad
            again = _attend(c, q, rows, kv)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype", list(PAGES))
@pytest.mark.parametrize("rows", [1, 40])
def test_attention_of_rows_that_are_not_finite(dtype, rows):
    """A row of NaN is alone with it; a score of +infinity makes NaN of its row, of -infinity takes the token out."""
    rng = np.random.default_rng(4)
    counts, kv = (rows,) * 4, (40 + rows,) * 4
    c = Cache(rng, dtype, 2, 64, kv, ([50], [0, 4]))
    q = rand(rng, (sum(counts), 4, 64), dtype)
    clean = _attend(c, q, counts, kv)
    bad = q.clone()
    bad[0, 1, 3] = float("nan")
    out, lse = _attend(c, bad, counts, kv)
    assert bool(out[0, 1].isnan().all()) and bool(lse[0, 1].isnan())
    out[0, 1], lse[0, 1] = clean[0][0, 1], clean[1][0, 1]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("dtype", list(PAGES))
def test_attention_scores_far_apart(dtype):
    """Scores of hundreds: one token has all the weight, and the maximum moves at the end, at the start, in between."""
    rng = np.random.default_rng(8)
    kv, rows = (300, 300, 300, 20), (1, 1, 1, 1)
    c = Cache(rng, dtype, 1, 128, kv, ([400], [0, 4]))
    q = rand(rng, (4, 4, 128), dtype, 8.0)
    c.k.mul_(4)
    page, slot = kv16.slots(c.table[0], 300)
    for at in (0, 150, 299):
        c.k[page[at], 0, slot[at]] = q[0, at % 4]
    _check_attention(c, q, rows, kv)


@pytest.mark.parametrize("dtype", list(PAGES))
def test_attention_weights_alike(dtype):
    """All scores 0: the mean of V, and lse the logarithm of the count, to far more tokens than a type can count."""
    rng = np.random.default_rng(9)
    n, p = 9001, 9000
    c = Cache(rng, dtype, 2, 64, [n, 5], ([p], [0, 2]))
    q = torch.zeros(2, 4, 64, dtype=PAGES[dtype], device="cuda")
    _, lse = _check_attention(c, q, (1, 1), (n, 5))
    np.testing.assert_allclose(lse.cpu().numpy()[0], np.log(n + p), rtol=1e-6)


def test_attention_does_not_depend_on_the_run_or_the_stream():
    rng = np.random.default_rng(10)
    kv, rows = [int(x) for x in rng.integers(1, 3000, 20)], (1,) * 20
    c = Cache(rng, "bf16", 4, 128, kv, ([2500], [0, 20]))
    q = rand(rng, (20, 28, 128), "bf16", 2.0)
    out, lse = _attend(c, q, rows, kv)
    side = torch.cuda.Stream()
    for _ in range(5):
        again = _attend(c, q, rows, kv, stream=side.cuda_stream)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    # two calls at once, each with a workspace of its own
    spaces = [c.new_workspace(28, 20) for _ in range(2)]
    outs = [torch.empty_like(out) for _ in range(2)]
    rs = ints(starts(rows))
    torch.cuda.synchronize()
    for w, o, st in zip(spaces, outs, (side, torch.cuda.Stream())):
        for _ in range(10):
            assert c.attention(q, rs, o, None, stream=st.cuda_stream, workspace=w) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


def test_attention_strided_rows_and_no_lse():
    rng = np.random.default_rng(11)
    kv, rows = (40, 500), (2, 3)
    c = Cache(rng, "f16", 2, 128, kv, ([77], [0, 2]))
    wide = rand(rng, (5, 12 + 7, 128), "f16", 2.0)
    q = wide[:, 3:15]
    ref, _ = _attend(c, q.contiguous(), rows, kv)
    out = torch.empty_like(ref)
    assert c.attention(q, ints(starts(rows)), out) == 0
    assert torch.equal(out, ref)


def test_attention_through_a_table_that_shares_pages():
    """Two sequences may read the same pages, and a prefix's pages may be a sequence's."""
    rng = np.random.default_rng(12)
    c = Cache(rng, "bf16", 2, 128, (100, 100), ([100], [0, 2]))
    c.table[1] = c.table[0]
    c.prefix[0][0] = c.table[0]
    c.dev_table, c.dev_prefix[0] = ints(c.table), ints(c.prefix[0])
    _check_attention(c, rand(rng, (4, 12, 128), "bf16"), (1, 3), (100, 100))


def test_attention_leaves_out_what_is_out_of_range():
    """Pages, lengths and groups that are not there: reported, and left out; the other sequences are as without them."""
    rng = np.random.default_rng(13)
    kv, rows = [200, 50, 60, 70], (1, 2, 1, 150)
    for rows in ((1, 2, 1, 1), (1, 2, 1, 60)):
        def fresh():
            r = np.random.default_rng(14)
            return Cache(r, "f16", 2, 64, kv, ([150, 40], [0, 2, 4])), rand(r, (sum(rows), 4, 64), "f16")
        c, q = fresh()
        good, _ = _attend(c, q, rows, kv)
        r = starts(rows)
        for change, others in (
                (lambda c: c.dev_table.__setitem__((0, 3), c.pages), slice(r[1], None)),
                (lambda c: c.dev_table.__setitem__((0, 3), -1), slice(r[1], None)),
                (lambda c: c.kv.__setitem__(1, -5), slice(r[2], None)),
                (lambda c: c.kv.__setitem__(1, 16 * c.dev_table.shape[1] + 1), slice(r[2], None)),
                (lambda c: c.dev_prefix[0].__setitem__((0, 2), 1 << 30), slice(r[2], None)),
                (lambda c: c.dev_prefix[1].__setitem__(1, -1), slice(0, r[2])),
                (lambda c: c.dev_prefix[1].__setitem__(1, 1 << 20), slice(0, r[2])),
                (lambda c: c.dev_prefix[2].__setitem__(2, 5), slice(0, r[2]))):
            c, q = fresh()
            change(c)
            out, lse = _attend(c, q, rows, kv, check_err=L.LLM_ERR_DEVICE)
            assert torch.equal(out[others], good[others])
            assert bool(out.isfinite().all())
        # a sequence whose length is out of range has no tokens of its own; behind no prefix its rows see nothing
        c, q = fresh()
        c.kv[1] = -5
        c.dev_prefix = None
        out, lse = _attend(c, q, rows, kv, check_err=L.LLM_ERR_DEVICE)
        assert bool((out[r[1]:r[2]] == 0).all()) and bool(lse[r[1]:r[2]].isneginf().all())


def test_attention_without_a_page_is_attention_without_its_tokens():
    rng = np.random.default_rng(15)
    c = Cache(rng, "bf16", 2, 128, (40,), ([48], [0, 1]))
    q = rand(rng, (1, 12, 128), "bf16")
    c.dev_table[0, 1] = -1
    c.dev_prefix[0][0, 0] = c.pages + 7
    out, lse = _attend(c, q, (1,), (40,), check_err=L.LLM_ERR_DEVICE)
    k, v = c.host()
    table, front = np.array([[c.table[0, 0], c.table[0, 2]]]), c.prefix[0][:, 1:]
    ref = kv16.attention(k, v, table, [0, 1], [24], as_f32(q), (front, [32], [0, 1]))
    tol, ltol = attention_bounds("bf16", *ref, 56)
    assert np.all(np.abs(as_f32(out) - ref[0]) <= tol) and np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)


# ---------------------------------------------------------------- weights


def _check_weigh(rng, dtype, Hq, Hkv, d, rows, kv, keep, extra=0):
    c = Cache(rng, dtype, Hkv, d, kv)
    n = sum(rows)
    q = rand(rng, (n + extra, Hq, d), dtype, 2.0)
    ref = kv16.attention(*c.host(), c.table, starts(rows), kv, as_f32(q[:n]))
    lse = np.full((n + extra, Hq), np.nan, np.float32)
    lse[:n] = ref[1]
    old = rng.random((len(kv), Hkv, max(kv) + 5)).astype(np.float32)
    scores = torch.from_numpy(old).cuda()
    new, size = kv16.weigh(c.host()[0], c.table, starts(rows), kv, as_f32(q[:n]), lse[:n], keep, old)
    assert c.weigh(q, ints(starts(rows)), torch.from_numpy(lse).cuda(), keep, scores) == 0
    got = scores.cpu().numpy()
    assert c.err.item() == 0
    bad = np.abs(got - new) / weigh_bounds(new, size, keep, old, max(rows) * Hq // Hkv)
    assert np.all(bad <= 1), (float(np.nanmax(bad)), np.argwhere(~(bad <= 1))[:4])
    for b, m in enumerate(kv):
        live = m if rows[b] else 0
        assert np.array_equal(got[b, :, live:], old[b, :, live:])
    return got


@pytest.mark.parametrize("dtype", list(PAGES))
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("rows,kv", [((1,), (1,)), ((1, 0, 1, 1), (16, 5, 17, 300)), ((5, 3, 4), (5, 100, 33)), ((130, 64), (130, 500)),
                                     ((1, 300), (1000, 300)), ((4, 1, 2), (2, 0, 2))])
def test_weigh(dtype, Hq, Hkv, d, rows, kv):
    _check_weigh(np.random.default_rng(Hq + sum(kv)), dtype, Hq, Hkv, d, rows, kv, 0.75, extra=2)


def test_weigh_adds_up_to_the_rows():
    """Each row's weights sum to one, however the rows are cut into calls."""
    rng = np.random.default_rng(16)
    for rows, kv in (((1, 1), (700, 90)), ((200, 30), (200, 77))):
        got = _check_weigh(rng, "bf16", 12, 2, 128, rows, kv, 0.0)
        total = np.array([got[b, :, :kv[b]].sum(-1) for b in range(2)])
        np.testing.assert_allclose(total, np.array(rows)[:, None] * 6 * np.ones((1, 2)), rtol=1e-4)


def test_weigh_forgets_without_looking():
    """keep 0 does not read what was there, tokens of the call start from nothing; lse of -infinity and NaN."""
    rng = np.random.default_rng(17)
    for rows in ((2, 2), (70, 2)):
        kv = (80, 60)
        c = Cache(rng, "f16", 2, 64, kv)
        q = rand(rng, (sum(rows), 4, 64), "f16")
        out, lse = _attend(c, q, rows, kv)
        a, b = (torch.full((2, 2, 90), x, device="cuda") for x in (float("nan"), 0.0))
        rs = ints(starts(rows))
        assert c.weigh(q, rs, lse, 0.0, a) == 0 and c.weigh(q, rs, lse, 1.0, b) == 0
        for i in range(2):
            assert torch.equal(a[i, :, :kv[i]], b[i, :, :kv[i]])
            assert bool(a[i, :, kv[i]:].isnan().all()) and bool((b[i, :, kv[i]:] == 0).all())
        lse[0] = float("-inf")
        x = torch.zeros(2, 2, 90, device="cuda")
        assert c.weigh(q, rs, lse, 0.0, x) == 0
        assert bool(x.isfinite().all()) and torch.equal(x[1], b[1])
        lse[0] = float("nan")
        assert c.weigh(q, rs, lse, 0.0, x) == 0
        first = kv[0] - rows[0] + 1  # what row 0 sees
        assert bool(x[0, :, :first].isnan().all()) and bool(x[0, :, first:kv[0]].isfinite().all()) and torch.equal(x[1], b[1])


def test_weigh_does_not_see_what_lies_behind_and_leaves_out_what_is_out_of_range():
    for rows in ((1, 2, 1), (1, 70, 1)):
        kv = (50, 77, 20)
        rng = np.random.default_rng(18)
        c = Cache(rng, "bf16", 2, 128, kv)
        q = rand(rng, (sum(rows), 12, 128), "bf16")
        out, lse = _attend(c, q, rows, kv)
        rs = ints(starts(rows))
        good = torch.zeros(3, 2, 80, device="cuda")
        assert c.weigh(q, rs, lse, 0.0, good) == 0
        seen = torch.zeros(c.pages, 16, dtype=torch.bool)
        for b, n in enumerate(kv):
            seen[kv16.slots(c.table[b], n)] = True
        c.k.permute(0, 2, 1, 3)[~seen.cuda()] = float("nan")
        x = torch.zeros_like(good)
        assert c.weigh(q, rs, lse, 0.0, x) == 0 and torch.equal(x, good)
        assert c.err.item() == 0
        keep_table = c.dev_table.clone()
        c.dev_table[1, 2] = c.pages
        assert c.weigh(q, rs, lse, 0.0, x) == 0
        assert c.err.item() == L.LLM_ERR_DEVICE
        assert torch.equal(x[0], good[0]) and torch.equal(x[2], good[2]) and torch.equal(x[1, :, :32], good[1, :, :32])
        assert torch.equal(x[1, :, 48:], good[1, :, 48:]) and bool((x[1, :, 32:48] == 0).all())
        c.dev_table = keep_table
        for n in (-3, 16 * c.dev_table.shape[1] + 1):
            c.err.zero_()
            x = torch.full_like(good, 3.0)
            assert c.weigh(q, rs, lse, 0.0, x, kv=ints([50, n, 20])) == 0
            assert c.err.item() == L.LLM_ERR_DEVICE and bool((x[1] == 3).all()) and torch.equal(x[0, :, :50], good[0, :, :50])
        c.err.zero_()
        short = torch.full((3, 2, 60), 3.0, device="cuda")  # a sequence longer than its scores
        assert c.weigh(q, rs, lse, 0.0, short) == 0
        assert c.err.item() == L.LLM_ERR_DEVICE and bool((short[1] == 3).all()) and torch.equal(short[0, :, :50], good[0, :, :50])


# ---------------------------------------------------------------- eviction


def _check_evict(rng, dtype, Hkv, d, kv, budget, first, last, scores, in_place, stride=None):
    c = Cache(rng, dtype, Hkv, d, kv)
    pools = [x.cpu().view(torch.int16).numpy().copy() for x in (c.k, c.v)]
    s = torch.from_numpy(scores).cuda()
    s_out = s if in_place else torch.full_like(s, -5.0)
    kept = torch.full((len(kv), Hkv, budget), -9, dtype=torch.int32, device="cuda")
    new = torch.zeros(len(kv), dtype=torch.int32, device="cuda")
    ref_out, ref_kept = (scores.copy() if in_place else np.full_like(scores, -5.0)), np.full(kept.shape, -9, np.int32)
    ref_len = kv16.evict(pools, c.table, np.array(kv), budget, first, last, scores, ref_out, ref_kept)
    assert c.evict(budget, first, last, s, s_out, kept, new) == 0
    assert c.err.item() == 0
    assert np.array_equal(new.cpu().numpy(), ref_len) and np.array_equal(kept.cpu().numpy(), ref_kept)
    assert np.array_equal(s_out.cpu().numpy(), ref_out, equal_nan=True)
    for x, ref in zip((c.k, c.v), pools):
        assert np.array_equal(x.cpu().view(torch.int16).numpy(), ref)


@pytest.mark.parametrize("dtype,Hkv,d", [("bf16", 2, 64), ("f16", 3, 128), ("bf16", 8, 128)])
@pytest.mark.parametrize("kv,budget,first,last", [
    ((1,), 1, 0, 0), ((2, 1, 0), 1, 0, 0), ((17, 16, 300), 16, 4, 4), ((100, 65, 64, 63), 64, 0, 64), ((90, 200), 64, 64, 0),
    ((1000, 5, 733), 100, 4, 32), ((4159,), 4096, 4, 512), ((5000, 4097), 300, 0, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(dtype, Hkv, d, kv, budget, first, last, in_place):
    rng = np.random.default_rng(sum(kv) + budget)
    scores = rng.random((len(kv), Hkv, max(kv) + 3)).astype(np.float32)
    _check_evict(rng, dtype, Hkv, d, kv, budget, first, last, np.ascontiguousarray(scores), in_place)


@pytest.mark.parametrize("kind", ["alike", "few values", "signs", "infinities and NaN", "near", "only NaN"])
def test_evict_scores(kind):
    """Ties go to the lower slot; all kinds of numbers."""
    rng = np.random.default_rng(19)
    kv, Hkv, budget = (900, 777, 1300), 2, 256
    shape = (3, Hkv, 1300)
    scores = {"alike": np.full(shape, 0.25), "few values": rng.integers(0, 4, shape), "signs": rng.standard_normal(shape) * (rng.random(shape) < 0.7),
              "infinities and NaN": rng.choice([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-45, 3e38, 1.0], shape),
              "near": 1.0 + rng.integers(0, 300, shape) * 2.0 ** -23, "only NaN": np.full(shape, np.nan)}[kind].astype(np.float32)
    for in_place in (False, True):
        _check_evict(rng, "bf16", Hkv, 64, kv, budget, 3, 20, scores.copy(), in_place)


def test_evict_more_tokens_than_shared_memory_holds():
    rng = np.random.default_rng(20)
    kv = (60000, 50001)
    scores = np.round(rng.random((2, 1, 60000)) * 5000).astype(np.float32)
    for in_place in (False, True):
        _check_evict(rng, "f16", 1, 64, kv, 20000, 4, 1000, scores.copy(), in_place)


def test_evict_leaves_out_what_is_out_of_range():
    rng = np.random.default_rng(21)
    kv = (100, 120, 90)
    c = Cache(rng, "bf16", 2, 64, kv)
    s = torch.rand(3, 2, 128, device="cuda")
    for bad in (-4, 16 * c.dev_table.shape[1] + 1, 129):
        c.err.zero_()
        kept, new = torch.full((3, 2, 50), -9, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
        before, out = [x.clone() for x in (c.k, c.v)], torch.zeros_like(s)
        wide = c if bad != 129 else None
        if wide is None:  # longer than its scores, not than its table
            c.dev_table = torch.cat([c.dev_table, c.dev_table[:, :1]], 1).contiguous()
        assert c.evict(50, 0, 0, s, out, kept, new, kv=ints([100, bad, 90])) == 0
        assert c.err.item() == L.LLM_ERR_DEVICE
        assert new.tolist() == [50, bad, 50] and bool((kept[1] == -9).all()) and bool((out[1] == 0).all()) and bool((kept[0] >= 0).all())
        for now, old in zip((c.k, c.v), before):
            mine = torch.from_numpy(c.table[1]).long()
            mine = mine[mine >= 0].cuda()
            assert torch.equal(now[mine], old[mine])
    # a page that is not there: its tokens are not moved, nor moved to; the others are
    c = Cache(rng, "bf16", 2, 64, kv)
    c.dev_table[0, 2] = c.pages
    before = [x.clone() for x in (c.k, c.v)]
    kept, new = torch.full((3, 2, 50), -9, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    assert c.evict(50, 0, 0, s, torch.zeros_like(s), kept, new) == 0
    assert c.err.item() == L.LLM_ERR_DEVICE
    for g in range(2):
        for x, old in zip((c.k, c.v), before):
            for j, i in enumerate(kept[0, g].tolist()):
                if i // 16 != 2 and j // 16 != 2:
                    assert torch.equal(x[c.table[0, j // 16], g, j % 16], old[c.table[0, i // 16], g, i % 16])


# ---------------------------------------------------------------- together


def _pipeline(dtype, steps, graph):
    """Prompts behind a shared prefix, then decode steps of sequences held to a budget: rotation into the pages, attention,
    weights, eviction; against the same steps of the oracle on what the kernels left in the pages."""
    rng = np.random.default_rng(22)
    B, Hq, Hkv, d, budget, prompt = 3, 12, 2, 128, 48, (60, 33, 50)
    axis, n_axes = _axes(d, "sections")
    capacity = [budget + 40] * B
    c = Cache(rng, dtype, Hkv, d, [0] * B, ([70], [0, B]), capacity=capacity)
    scores, lens = torch.zeros(B, Hkv, budget + 40, device="cuda"), ints([0] * B)
    kept = torch.zeros(B, Hkv, budget, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    seen = [int(x) for x in [0] * B]  # positions so far
    results = []
    for step in range(steps):
        rows = prompt if step == 0 else (1,) * B
        n = sum(rows)
        qkv = rand(rng, (n, (Hq + 2 * Hkv) * d), "f32", 1.5)
        pos = np.concatenate([70 + seen[b] + np.arange(rows[b]) for b in range(B)])
        seen = [s + r for s, r in zip(seen, rows)]
        pos3 = ints(np.stack([pos, pos + 3, pos * 2]))
        rs, add = ints(starts(rows)), ints(rows)
        q = torch.empty(n, Hq, d, dtype=PAGES[dtype], device="cuda")
        out, lse = torch.empty_like(q), torch.empty(n, Hq, device="cuda")
        c.workspace = None
        c.workspace = c.new_workspace(Hq, n)
        torch.cuda.synchronize()
        run_kv = (lens + add).int()

        def call(stream=None):
            assert c.rope_append(qkv, Hq, None, axis, n_axes, pos3, rs, q, kv=run_kv, stream=stream) == 0
            assert c.attention(q, rs, out, lse, kv=run_kv, stream=stream) == 0
            assert c.weigh(q, rs, lse, 1.0, scores, kv=run_kv, stream=stream) == 0
            assert c.evict(budget, 4, 16, scores, scores, kept, new, kv=run_kv, stream=stream) == 0

        if graph:
            side = torch.cuda.Stream()
            g = torch.cuda.CUDAGraph()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(g, stream=side):
                call(side.cuda_stream)
            g.replay()
        else:
            call()
        torch.cuda.synchronize()
        assert c.err.item() == 0
        lens = new.clone()
        results.append([x.clone() for x in (q, out, lse, scores[..., :budget], kept, new, c.k, c.v)])
    return results


@pytest.mark.parametrize("dtype", list(PAGES))
def test_steps_together_eager_and_in_graphs(dtype):
    for x, y in zip(_pipeline(dtype, 30, False), _pipeline(dtype, 30, True)):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_steps_together_against_the_oracle():
    """One long prompt and twelve steps, everything followed in 64 bits from what the kernels wrote into the pages."""
    rng = np.random.default_rng(23)
    B, Hq, Hkv, d, budget = 2, 4, 2, 64, 40
    axis, n_axes = _axes(d, "sections")
    c = Cache(rng, "bf16", Hkv, d, [0] * B, ([37], [0, B]), capacity=[100] * B)
    lens = np.zeros(B, int)
    scores = torch.zeros(B, Hkv, 100, device="cuda")
    kept, new = torch.zeros(B, Hkv, budget, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    for step in range(13):
        rows = (70, 45) if step == 0 else (1, 2)
        n, kv = sum(rows), lens + np.array(rows)
        qkv = rand(rng, (n, (Hq + 2 * Hkv) * d), "bf16", 1.5)
        pos = rng.integers(0, 3000, (3, n)).astype(np.int32)
        q = torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda")
        out, lse, rs, dkv = torch.empty_like(q), torch.empty(n, Hq, device="cuda"), ints(starts(rows)), ints(kv)
        c.workspace = None
        assert c.rope_append(qkv, Hq, None, axis, n_axes, ints(pos), rs, q, kv=dkv) == 0
        assert c.attention(q, rs, out, lse, kv=dkv) == 0
        k, v = c.host()
        ref = kv16.attention(k, v, c.table, starts(rows), kv, as_f32(q), c.prefix)
        tol, ltol = attention_bounds("bf16", *ref, max(kv) + 37)
        assert np.all(np.abs(as_f32(out) - ref[0]) <= tol) and np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)
        old = scores.cpu().numpy()
        assert c.weigh(q, rs, lse, 1.0, scores, kv=dkv) == 0
        want, size = kv16.weigh(k, c.table, starts(rows), kv, as_f32(q), lse.cpu().numpy(), 1.0, old)
        now = scores.cpu().numpy()
        assert np.all(np.abs(now - want) <= weigh_bounds(want, size, 1.0, old, max(rows) * 2))
        pools = [x.cpu().view(torch.int16).numpy().copy() for x in (c.k, c.v)]
        ref_kept, ref_scores = kept.cpu().numpy(), now.copy()
        ref_len = kv16.evict(pools, c.table, kv, budget, 4, 8, now, ref_scores, ref_kept)
        assert c.evict(budget, 4, 8, scores, scores, kept, new, kv=dkv) == 0
        assert np.array_equal(kept.cpu().numpy(), ref_kept) and np.array_equal(scores.cpu().numpy(), ref_scores)
        assert all(np.array_equal(x.cpu().view(torch.int16).numpy(), p) for x, p in zip((c.k, c.v), pools))
        lens = np.array(new.tolist())
        assert np.array_equal(lens, ref_len)
    assert c.err.item() == 0
