"""Helpers for the 16-bit K/V cache tests: a cache on the device, its calls, and bounds on their errors."""
import ctypes

import numpy as np
import torch

from quantized_decode_gb300 import _lib as L

from ._kv8 import DTYPES, as_f32, ints, page_table, starts  # noqa: F401

PAGES = {"f16": torch.float16, "bf16": torch.bfloat16}
HEADS = [(4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128), (3, 3, 64), (8, 1, 128), (5, 1, 64)]


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DTYPES[dtype][0]).cuda()


class Cache:
    """Pools of random numbers, sequences of these lengths and prefixes (lengths, seq_start) on shuffled pages."""

    def __init__(self, rng, dtype, Hkv, d, kv_len, prefix=None, capacity=None, extra=3):
        lens = list(capacity if capacity is not None else kv_len)
        both, pages = page_table(rng, lens + (list(prefix[0]) if prefix else []), extra)
        self.dtype, self.d, self.Hkv, self.pages = dtype, d, Hkv, pages
        self.k, self.v = (rand(rng, (pages, Hkv, 16, d), dtype) for _ in range(2))
        n = len(lens)
        self.table = np.ascontiguousarray(both[:n, :max(1, max(-(-x // 16) for x in lens))])
        self.dev_table, self.kv = ints(self.table), ints(kv_len)
        self.prefix = self.dev_prefix = None
        if prefix:
            own = np.ascontiguousarray(both[n:, :max(1, max(-(-x // 16) for x in prefix[0]))])
            self.prefix = (own, list(prefix[0]), list(prefix[1]))
            self.dev_prefix = [ints(x) for x in self.prefix]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = None

    def struct(self, **kw):
        f = dict(dtype=DTYPES[self.dtype][1], n_kv_heads=self.Hkv, head_dim=self.d, n_pool_pages=self.pages, k_pool=self.k.data_ptr(),
                 v_pool=self.v.data_ptr(), page_table=self.dev_table.data_ptr(), n_seqs=self.dev_table.shape[0],
                 table_stride=self.dev_table.shape[1])
        return ctypes.byref(L.llm_kv16_cache(**{**f, **kw}))

    def prefix_struct(self):
        if self.dev_prefix is None:
            return None
        t, n, s = self.dev_prefix
        return ctypes.byref(L.llm_kv16_prefix(page_table=t.data_ptr(), len=n.data_ptr(), seq_start=s.data_ptr(), n_groups=n.shape[0],
                                              table_stride=t.shape[1]))

    def host(self):
        return as_f32(self.k), as_f32(self.v)

    def rope_append(self, qkv, Hq, gains, axis, n_axes, pos, row_start, q_out, eps=1e-6, base=1e6, kv=None, stream=None, n_rows=None):
        n, width = qkv.shape
        size, d = qkv.element_size(), self.d
        name = next(k for k, v in DTYPES.items() if v[0] == qkv.dtype)
        at = qkv.data_ptr()
        axes = (ctypes.c_uint8 * (d // 2))(*[int(x) for x in axis])
        g = [None, None] if gains is None else [x.data_ptr() for x in gains]
        return L.load().llm_op_kv16_rope_append(
            self.struct(), DTYPES[name][1], at, width, at + Hq * d * size, width, at + (Hq + self.Hkv) * d * size, width, *g, eps, base, axes,
            n_axes, pos.data_ptr(), row_start.data_ptr(), (self.kv if kv is None else kv).data_ptr(), n if n_rows is None else n_rows, Hq,
            q_out.data_ptr(), self.err.data_ptr(), stream)

    def new_workspace(self, Hq, rows):
        need = ctypes.c_int64()
        L.check(L.load().llm_op_kv16_attention_workspace(self.struct(), self.prefix_struct(), Hq, rows, ctypes.byref(need)), "workspace")
        return torch.zeros(need.value, dtype=torch.uint8, device="cuda")

    def attention(self, q, row_start, out, lse=None, kv=None, stream=None, workspace=None):
        Hq = out.shape[1]
        if workspace is None:
            if self.workspace is None:
                self.workspace = self.new_workspace(Hq, q.shape[0])
            workspace = self.workspace
        return L.load().llm_op_kv16_attention(
            self.struct(), self.prefix_struct(), q.data_ptr(), q.stride(0), row_start.data_ptr(), (self.kv if kv is None else kv).data_ptr(),
            q.shape[0], Hq, out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
            self.err.data_ptr(), stream)

    def weigh(self, q, row_start, lse, keep, scores, kv=None, stream=None):
        return L.load().llm_op_kv16_weigh(
            self.struct(), q.data_ptr(), q.stride(0), row_start.data_ptr(), (self.kv if kv is None else kv).data_ptr(), q.shape[0], q.shape[1],
            lse.data_ptr(), keep, scores.data_ptr(), scores.stride(1), self.err.data_ptr(), stream)

    def evict(self, budget, n_first, n_last, scores, scores_out, kept, new_len, kv=None, stream=None):
        return L.load().llm_op_kv16_evict(
            self.struct(), (self.kv if kv is None else kv).data_ptr(), budget, n_first, n_last, scores.data_ptr(), scores_out.data_ptr(),
            scores.stride(1), kept.data_ptr(), new_len.data_ptr(), self.err.data_ptr(), stream)


def attention_bounds(dtype, out, lse, absv, absqk, kv):
    """How far out and lse may be from the 64-bit ones, from the arithmetic of the operator:

    A score is a sum of d exact products in fp32: at most 32 additions, each off by 2^-23 of the sum of magnitudes if it
    truncates, and a few products of 2^-24: 36 * 2^-23 * A with A = sum |q_i k_i| / sqrt(d).  exp2 adds 2^-22: a weight is off by
    e = A 36 2^-23 + 2^-21 of itself, the output by 2 e of sum w|v| (numerator and denominator), and by its own
    additions: kv / 16 steps and 400 joined parts at most, 2^-23 of sum w|v| each.  Weights are rounded to the pages' type once,
    half a step of each (bf16 2^-8, fp16 2^-11; the least fp16 ones by 2^-25 2^-7 at most, next to a largest of 1, where all of
    them together stay below 2^-11 of the sum up to 2^20 tokens), and the result once more (at least 2^-25 in fp16).
    lse: the scores' absolute error, 2^-22 of itself and 2^-20 for the sum and its logarithm."""
    half = torch.finfo(DTYPES[dtype][0]).eps / 2
    e = absqk[..., None] * 36 * 2.0 ** -23 + 2.0 ** -21
    tol = absv * (2 * e + (kv / 16 + 400) * 2.0 ** -23 + half) + np.abs(out) * half + 2.0 ** -25 * (dtype == "f16")
    return tol + 1e-30, absqk * 36 * 2.0 ** -23 + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22 + 2.0 ** -20


def weigh_bounds(new, size, keep, old, terms):
    """Each term is off by its exponent's absolute error, (A + |lse|) 36 2^-23, and 2^-20 for exp2 and the products of
    log2(e): size holds term * (A + |lse| + 1).  A sum of `terms` of them in fp32: each addition 2^-24 of the sum so far."""
    return size * 44 * 2.0 ** -23 + np.abs(new) * (terms + 2) * 2.0 ** -24 + keep * np.abs(old) * 2.0 ** -23 + 1e-37
