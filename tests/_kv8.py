"""Helpers for the 8-bit K/V cache tests: a cache in numpy and its copy on the device."""
import ctypes

import numpy as np
import torch

from oracle import kv8
from quantized_decode_gb300 import _lib as L

DTYPES = {"f32": (torch.float32, L.LLM_DTYPE_F32), "f16": (torch.float16, L.LLM_DTYPE_F16), "bf16": (torch.bfloat16, L.LLM_DTYPE_BF16)}
FORMATS = {"int8": L.LLM_KV8_INT8, "e4m3": L.LLM_KV8_E4M3}


def host_cache(rng, fmt, pages, Hkv, d):
    """Random codes of the whole range and scales that differ by page and head."""
    cache = {"fmt": fmt}
    for x in ("k", "v"):
        codes = kv8.encode(rng.standard_normal((pages, Hkv, 16, d)).astype(np.float32) * (kv8.CODE_MAX[fmt] / np.float32(3.5)), fmt)
        cache[x] = codes
        cache[x + "s"] = ((0.75 + rng.random((pages, Hkv))) * 3.5 / float(kv8.CODE_MAX[fmt])).astype(np.float32)
    return cache


def page_table(rng, kv_len, extra=3, capacity=None):
    """Shuffled pages for sequences of these lengths (at capacity[b] tokens each): table, pages in the pools.  Entries behind
    a sequence's pages name no page."""
    need = [-(-int(n) // 16) for n in (capacity if capacity is not None else kv_len)]
    total = sum(need) + extra
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(need), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


class DeviceCache:
    def __init__(self, cache, table):
        self.fmt = cache["fmt"]
        self.shape = cache["k"].shape
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.k, self.v, self.ks, self.vs, self.table = up(cache["k"]), up(cache["v"]), up(cache["ks"]), up(cache["vs"]), up(table)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = None

    def struct(self):
        pages, Hkv, _, d = self.shape
        return ctypes.byref(L.llm_kv8_cache(
            format=FORMATS[self.fmt], n_kv_heads=Hkv, head_dim=d, n_pool_pages=pages, k_codes=self.k.data_ptr(),
            v_codes=self.v.data_ptr(), k_scale=self.ks.data_ptr(), v_scale=self.vs.data_ptr(),
            page_table=self.table.data_ptr(), n_seqs=self.table.shape[0], table_stride=self.table.shape[1]))

    def host(self):
        return {"fmt": self.fmt, "k": self.k.cpu().numpy(), "v": self.v.cpu().numpy(), "ks": self.ks.cpu().numpy(),
                "vs": self.vs.cpu().numpy()}

    def append(self, dtype, k, v, row_start, kv_len, n_rows=None, stream=None):
        return L.load().llm_op_kv8_append(self.struct(), DTYPES[dtype][1], k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0),
                                          row_start.data_ptr(), kv_len.data_ptr(), k.shape[0] if n_rows is None else n_rows,
                                          self.err.data_ptr(), stream)

    def read(self, dtype, k, v, row_start, kv_len, stream=None):
        return L.load().llm_op_kv8_read(self.struct(), DTYPES[dtype][1], row_start.data_ptr(), kv_len.data_ptr(), k.shape[0],
                                        k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), self.err.data_ptr(), stream)

    def attention(self, dtype, q, row_start, kv_len, out, lse=None, stream=None, workspace=None):
        lib, Hq = L.load(), out.shape[1]
        if workspace is None:
            if self.workspace is None:
                self.workspace = new_workspace(self, Hq, q.shape[0])
            workspace = self.workspace
        return lib.llm_op_kv8_attention(self.struct(), DTYPES[dtype][1], q.data_ptr(), q.stride(0), row_start.data_ptr(),
                                        kv_len.data_ptr(), q.shape[0], Hq, out.data_ptr(),
                                        None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                        self.err.data_ptr(), stream)


def new_workspace(cache, Hq, rows):
    need = ctypes.c_int64()
    L.check(L.load().llm_op_kv8_attention_workspace(cache.struct(), Hq, rows, ctypes.byref(need)), "workspace")
    return torch.zeros(need.value, dtype=torch.uint8, device="cuda")


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def as_f32(t):
    return t.float().cpu().numpy()


def attention_bounds(dtype, out, lse, absv, sumv, absqk, kv):
    """How far out and lse may be from the 64-bit ones, from the arithmetic of the operator:

    A score is a sum of d products of q's 22 bits (2^-22 of |q| for what the second fp16 half rounds off) in fp32: at most
    32 additions, each off by 2^-23 of the sum of magnitudes if it truncates, then 3 products of 2^-24: 36 * 2^-23 * A with
    A = sum |q_i k_i| / sqrt(d).  exp2 adds 2^-22, the split weights 2^-22: a weight is off by e = A 36 2^-23 + 2^-21 of itself,
    the output by 2 e of sum w|v| (numerator and denominator), and by its own additions: at most kv / 16 pages and 400 joined
    parts, 2^-23 of sum w|v| each.  A weight is also a pair of fp16 numbers, which have no spacing below 2^-24: next to a
    largest weight of 1 or more, the smallest are off by up to 2^-25 for 16-bit rows and by 2^-32 for fp32 ones (which are
    lifted by 2^7 at least before they are rounded), whatever their own size.  16-bit rows: products with fp16 weights of 11 bits, 2^-11 of sum w|v|, and the rounding of
    the result, half a step (2^-25 at least in fp16).  lse: the scores' absolute error, plus 2^-22 of itself and 2^-21 for the logarithm of the sum."""
    e = absqk[..., None] * 36 * 2.0 ** -23 + 2.0 ** -21
    tol = absv * (2 * e + (kv / 16 + 400) * 2.0 ** -23) + sumv * 2.0 ** (-32 if dtype == "f32" else -25)
    if dtype != "f32":
        tol = tol + absv * 2.0 ** -11 + np.abs(out) * torch.finfo(DTYPES[dtype][0]).eps / 2 + 2.0 ** -25 * (dtype == "f16")
    return tol + 1e-30, absqk * 36 * 2.0 ** -23 + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22 + 2.0 ** -20
