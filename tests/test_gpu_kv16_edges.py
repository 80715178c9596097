"""The 16-bit K/V cache operators where their kernels change course: clusters, lines of work, far pages, many sequences, numbers
that are out of order (GPU required)."""
import numpy as np
import pytest
import torch

from oracle import kv16
from quantized_decode_gb300 import _lib as L

from ._kv16 import Cache, as_f32, attention_bounds, ints, rand, starts, weigh_bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    L.load()


def _attend(c, q, rs, **kw):
    out, lse = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda"), torch.full(q.shape[:2], 55.0, device="cuda")
    assert c.attention(q, rs, out, lse, **kw) == 0
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d,rows,kv", [(12, 2, 128, (500, 420), (500, 700)), (28, 4, 128, (700, 3), (900, 5)), (8, 1, 64, (300,), (300,)),
                                              (5, 1, 64, (1000, 1), (1100, 400))])
def test_weigh_of_long_prompts(dtype, Hq, Hkv, d, rows, kv):
    """As many rows as make clusters share a block of tokens; a sequence of a few rows beside them."""
    rng = np.random.default_rng(Hq)
    c = Cache(rng, dtype, Hkv, d, kv)
    q = rand(rng, (sum(rows) + 1, Hq, d), dtype, 2.0)
    ref = kv16.attention(*c.host(), c.table, starts(rows), kv, as_f32(q[:-1]))
    lse = np.concatenate([ref[1], np.full((1, Hq), np.nan)]).astype(np.float32)
    old = rng.random((len(kv), Hkv, max(kv) + 5)).astype(np.float32)
    for keep in (0.0, 1.0):
        scores = torch.from_numpy(old.copy()).cuda()
        new, size = kv16.weigh(c.host()[0], c.table, starts(rows), kv, as_f32(q[:-1]), lse[:-1], keep, old)
        first = None
        for _ in range(3):
            scores.copy_(torch.from_numpy(old))
            assert c.weigh(q, ints(starts(rows)), torch.from_numpy(lse).cuda(), keep, scores) == 0
            first = scores.clone() if first is None else first
            assert torch.equal(scores, first)
        bad = np.abs(scores.cpu().numpy() - new) / weigh_bounds(new, size, keep, old, max(rows) * Hq // Hkv)
        assert np.all(bad <= 1), float(np.nanmax(bad))
    assert c.err.item() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_on_a_line_of_work(dtype):
    """Units of many lengths end to end: groups of prompts, prompts of no group, a prefix of one token."""
    rng = np.random.default_rng(31)
    rows = (200, 70, 1, 333, 90, 64)
    kv = (200, 900, 1, 500, 91, 64)
    c = Cache(rng, dtype, 8, 64, kv, ([1000, 1, 259], [0, 2, 3, 5]))
    q = rand(rng, (sum(rows), 32, 64), dtype, 2.0)
    rs = ints(starts(rows))
    out, lse = _attend(c, q, rs)
    ref = kv16.attention(*c.host(), c.table, starts(rows), kv, as_f32(q), c.prefix)
    tol, ltol = attention_bounds(dtype, *ref, 1900)
    assert np.all(np.abs(as_f32(out) - ref[0]) <= tol) and np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)
    assert c.err.item() == 0
    for _ in range(3):
        again = _attend(c, q, rs)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("prefix", [None, ([64, 200], [0, 500, 1000])])
def test_attention_and_weigh_of_a_thousand_sequences(prefix):
    rng = np.random.default_rng(32)
    B = 1000
    kv = [int(x) for x in rng.integers(1, 60, B)]
    rows = [1] * B
    c = Cache(rng, "bf16", 2, 64, kv, prefix)
    q = rand(rng, (B, 4, 64), "bf16", 2.0)
    out, lse = _attend(c, q, ints(starts(rows)))
    ref = kv16.attention(*c.host(), c.table, starts(rows), kv, as_f32(q), c.prefix)
    tol, ltol = attention_bounds("bf16", *ref, 300)
    assert np.all(np.abs(as_f32(out) - ref[0]) <= tol) and np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)
    old = np.zeros((B, 2, 64), np.float32)
    scores = torch.from_numpy(old).cuda()
    assert c.weigh(q, ints(starts(rows)), lse, 0.0, scores) == 0
    new, size = kv16.weigh(c.host()[0], c.table, starts(rows), kv, as_f32(q), lse.cpu().numpy(), 0.0, old)
    assert np.all(np.abs(scores.cpu().numpy() - new) <= weigh_bounds(new, size, 0.0, old, 2))
    assert c.err.item() == 0


@pytest.mark.parametrize("prefix", [None, ([90], [0, 14])])
def test_drafts_among_steps(prefix):
    """A few sequences with many rows among many with one: several tiles of rows in the kernel for few."""
    rng = np.random.default_rng(37)
    rows = (6, 1, 1, 1, 0, 1, 9, 1, 1, 1, 1, 0, 1, 1)
    kv = (40, 17, 300, 1, 9, 64, 2000, 5, 90, 31, 32, 0, 700, 8)
    for dtype, Hq, Hkv, d in (("bf16", 12, 4, 128), ("f16", 8, 2, 64)):
        c = Cache(rng, dtype, Hkv, d, kv, prefix)
        q = rand(rng, (sum(rows), Hq, d), dtype, 2.0)
        out, lse = _attend(c, q, ints(starts(rows)))
        ref = kv16.attention(*c.host(), c.table, starts(rows), kv, as_f32(q), c.prefix)
        tol, ltol = attention_bounds(dtype, *ref, 2100)
        assert np.all(np.abs(as_f32(out) - ref[0]) <= tol) and np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)
        old = rng.random((len(kv), Hkv, 2000)).astype(np.float32)
        scores = torch.from_numpy(old.copy()).cuda()
        assert c.weigh(q, ints(starts(rows)), lse, 1.0, scores) == 0
        # lse holds the prefix's weight too
        new, size = kv16.weigh(c.host()[0], c.table, starts(rows), kv, as_f32(q), lse.cpu().numpy(), 1.0, old)
        assert np.all(np.abs(scores.cpu().numpy() - new) <= weigh_bounds(new, size, 1.0, old, 9 * Hq // Hkv))
        assert c.err.item() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [(3, 1, 1, 1, 1, 1, 1, 1, 1), (40,), (300,)])
def test_a_key_that_is_not_finite_and_a_row_does_not_see(dtype, rows):
    """NaN and infinities in the key of a sequence's last token are the business of its last row alone."""
    rng = np.random.default_rng(38)
    kv = tuple(r + 50 for r in rows)
    for prefix in (None, ([70], [0, len(rows)])):
        c = Cache(rng, dtype, 2, 64, kv, prefix)
        q, rs = rand(rng, (sum(rows), 4, 64), dtype), ints(starts(rows))
        out, lse = _attend(c, q, rs)
        page, slot = (int(x[-1]) for x in kv16.slots(c.table[0], kv[0]))
        for bad in (float("nan"), float("inf")):
            c.k[page, :, slot] = bad
            got, glse = _attend(c, q, rs)
            keep = [i for i in range(sum(rows)) if i != rows[0] - 1]
            assert torch.equal(got[keep], out[keep]) and torch.equal(glse[keep], lse[keep])
            assert bool(got[rows[0] - 1].isnan().all())


def test_far_pages():
    """Pools of more than 2^32 bytes: the same tokens far up in them give the same results."""
    rng = np.random.default_rng(33)
    Hq, Hkv, d, far = 32, 8, 128, 140000
    kv, rows, prefix = (100, 40), (2, 1), ([77], [0, 2])
    c = Cache(rng, "bf16", Hkv, d, kv, prefix, extra=0)
    big = [torch.zeros(far + c.pages, Hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    big[0][far:], big[1][far:] = c.k, c.v
    q, rs = rand(rng, (3, Hq, d), "bf16", 2.0), ints(starts(rows))
    wide = rand(rng, (240, Hq, d), "bf16", 2.0)
    small = [_attend(c, q, rs)]
    scores = [torch.zeros(2, Hkv, 300, device="cuda") for _ in range(2)]
    assert c.weigh(q, rs, small[0][1], 0.0, scores[0]) == 0
    wide_rs, c.workspace = ints([0, 70, 100]), None
    small.append(_attend(c, wide, wide_rs))
    kept, new = torch.zeros(2, Hkv, 50, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    pages = c.k, c.v
    c.k, c.v, c.pages, c.workspace = big[0], big[1], far + c.pages, None
    c.dev_table = torch.where(c.dev_table >= 0, c.dev_table + far, c.dev_table)
    c.dev_prefix[0] = torch.where(c.dev_prefix[0] >= 0, c.dev_prefix[0] + far, c.dev_prefix[0])
    for got, ref in zip(_attend(c, q, rs), small[0]):
        assert torch.equal(got, ref)
    assert c.weigh(q, rs, small[0][1], 0.0, scores[1]) == 0 and torch.equal(scores[0], scores[1])
    c.workspace = None
    for got, ref in zip(_attend(c, wide, wide_rs), small[1]):
        assert torch.equal(got[:100], ref[:100])
    assert c.evict(50, 2, 10, scores[1], scores[1], kept, new) == 0
    qkv = rand(rng, (2, (Hq + 2 * Hkv) * d), "f32")
    at = torch.empty(2, Hq, d, dtype=torch.bfloat16, device="cuda")
    assert c.rope_append(qkv, Hq, None, np.zeros(d // 2, int), 1, ints([[1, 2]]), ints([0, 1, 2]), at, kv=ints([51, 41])) == 0
    torch.cuda.synchronize()
    assert c.err.item() == 0
    for x, mine, z in ((big[0], pages[0], 0), (big[1], pages[1], 1)):
        assert not bool(x[:far].any())
        for g in range(Hkv):
            table = c.table[0]
            for j, i in list(enumerate(kept[0, g].tolist()))[:48]:
                assert torch.equal(x[far + table[j // 16], g, j % 16], mine[table[i // 16], g, i % 16])


def test_numbers_out_of_order():
    """A row_start that falls, or leaves the rows, is reported; nothing outside the call's arrays is touched."""
    rng = np.random.default_rng(34)
    Hq, Hkv, d, n = 12, 2, 64, 300
    for kind in ([0, 200, 20, 290, 40, 300], [0, 300, 0, 300, 0, 300], [-5, 10, 20, 30, 40, 50], [0, 10, 500, 20, 30, 40]):
        kv = [64, 100, 300, 40, 20]
        c = Cache(rng, "f16", Hkv, d, kv, ([100, 40], [0, 2, 5]))
        guard = torch.full((n + 64, Hq, d), 5.0, dtype=torch.float16, device="cuda")
        q = rand(rng, (n, Hq, d), "f16")
        lse = torch.zeros(n, Hq, device="cuda")
        for rows in (n, 200):  # many rows, and (below) few
            c.err.zero_()
            c.workspace = None
            assert c.attention(q[:rows], ints(kind), guard[:rows], lse) == 0
            torch.cuda.synchronize()
            assert c.err.item() == L.LLM_ERR_DEVICE and bool((guard[n:] == 5).all())
            scores = torch.full((5, Hkv, 320), 3.0, device="cuda")
            c.err.zero_()
            assert c.weigh(q[:rows], ints(kind), lse, 1.0, scores) == 0
            torch.cuda.synchronize()
            assert c.err.item() == L.LLM_ERR_DEVICE and bool((scores[:, :, 304:] == 3).all())
        few = [min(max(x, -5), 30) for x in kind]
        c.err.zero_()
        c.workspace = None
        assert c.attention(q[:30], ints(few), guard[:30], lse) == 0
        assert c.weigh(q[:30], ints(few), lse, 1.0, scores) == 0
        qkv = rand(rng, (n, (Hq + 2 * Hkv) * d), "f32")
        assert c.rope_append(qkv, Hq, None, np.zeros(d // 2, int), 1, ints(np.arange(n)[None]), ints(kind), guard[:n]) == 0
        torch.cuda.synchronize()
        assert c.err.item() == L.LLM_ERR_DEVICE and bool((guard[n:] == 5).all())


def test_one_workspace_for_calls_of_many_kinds():
    """A workspace made for the largest call serves all, in any order, and is ready after each."""
    rng = np.random.default_rng(35)
    kv = [300, 20, 500]
    c = Cache(rng, "bf16", 2, 128, kv, ([400], [0, 3]))
    q = rand(rng, (400, 12, 128), "bf16", 2.0)
    space = c.new_workspace(12, 400)
    prefix = c.dev_prefix
    calls = [([1, 1, 1], True), ([150, 20, 230], True), ([1, 1, 1], False), ([5, 0, 3], True), ([200, 20, 100], False), ([0, 0, 1], True)]
    refs = []
    for rows, shared in calls * 3:
        c.dev_prefix = prefix if shared else None
        n = sum(rows)
        got = _attend(c, q[:n], ints(starts(rows)), workspace=space)
        c.workspace = None
        ref = _attend(c, q[:n], ints(starts(rows)))
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        refs.append(got)
    assert c.err.item() == 0
    for x, y in zip(refs[:6], refs[6:]):
        assert torch.equal(x[0], y[0])


def test_graphs_that_run_at_the_same_time():
    """Two captured steps with workspaces of their own, replayed on two streams, and one captured step replayed many times."""
    rng = np.random.default_rng(36)
    kv, rows = [700, 64, 900], (1, 1, 1)
    c = Cache(rng, "bf16", 2, 128, kv, ([1500], [0, 3]))
    q, rs = rand(rng, (3, 12, 128), "bf16", 2.0), ints(starts(rows))
    ref = _attend(c, q, rs)
    scores0 = torch.zeros(3, 2, 900, device="cuda")
    assert c.weigh(q, rs, ref[1], 0.0, scores0) == 0
    graphs = []
    for _ in range(2):
        space, out, lse, scores = c.new_workspace(12, 3), torch.zeros_like(ref[0]), torch.zeros_like(ref[1]), torch.zeros_like(scores0)
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            assert c.attention(q, rs, out, lse, stream=s.cuda_stream, workspace=space) == 0
            assert c.weigh(q, rs, lse, 0.0, scores, stream=s.cuda_stream) == 0
        graphs.append((g, s, out, lse, scores, space))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, *_x in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _g, _s, out, lse, scores, _w in graphs:
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1]) and torch.equal(scores, scores0)
    assert c.err.item() == 0
