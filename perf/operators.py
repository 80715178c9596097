"""What the 8-bit K/V cache operators are measured on: the q/k norm with the rotation, the quantising
cache write, the read back, and attention over the cache.

Each case is one call of one operator (``op``):

  rope    RMS norm of every query and key head and the rotation to its position
  write   rows of K and V quantised into the pages of their sequences, one scale for each page and head
  read    tokens of the cache back as dense rows
  attend  causal grouped-query attention of each sequence's last rows over its pages

``run`` computes them in plain torch while ``own`` is false and calls the library's entry points
(include/llm_ops.h) while it is true.  Shapes: ``hq`` query and ``hkv`` key/value heads of ``d``, ``seqs``
sequences, ``rows`` new rows in each (spread evenly around that number), ``kv`` tokens in the longest
sequence with those rows in it.
"""
import math

import torch

own = False

PAGE = 16
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPE_IDS = {"f32": 0, "f16": 1, "bf16": 2}
FORMATS = {"int8": 1, "e4m3": 2}
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}
HEADS = ((4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128))


def listed():
    def case(name, op, heads, **kw):
        hq, hkv, d = heads
        return {"name": name, "op": op, "hq": hq, "hkv": hkv, "d": d, **kw}

    tiny, m15, m7, m8 = HEADS
    return [
        # one decode step of one sequence: a single row, where only latency counts
        case("rope-step", "rope", m8, rows=1, dtype="f32", norm=True, far=4096),
        # a long prompt's rows at once, far into a long document
        case("rope-prompt", "rope", m8, rows=8191, dtype="bf16", norm=True, far=1 << 20),
        # the decode step of eight sequences that decode together: one token each into half-full pages
        case("write-step", "write", m7, seqs=8, rows=1, kv=4096, even=False, dtype="f32", fmt="int8"),
        # prompts of several users written at once, the last pages ragged
        case("write-prompts", "write", m8, seqs=8, rows=2000, kv=4000, even=False, dtype="bf16", fmt="e4m3"),
        # one short sequence read back, to move it to another cache
        case("read-one", "read", m15, seqs=1, rows=511, kv=511, even=True, dtype="bf16", fmt="e4m3"),
        # eight sequences read back whole, as a prefix cache hands them out
        case("read-many", "read", m7, seqs=8, rows=16000, kv=16000, even=False, dtype="f32", fmt="int8"),
        # the first tokens of a conversation on the smallest decoder: latency alone
        case("attend-first", "attend", tiny, seqs=1, rows=1, kv=17, even=True, dtype="f32", fmt="int8"),
        # one decode step at the engine's default context, fp32 rows as the engine keeps them
        case("attend-step", "attend", m7, seqs=1, rows=1, kv=4096, even=True, dtype="f32", fmt="int8"),
        # eight sequences of very different lengths decoding together
        case("attend-batch", "attend", m8, seqs=8, rows=1, kv=32768, even=False, dtype="bf16", fmt="e4m3"),
        # long documents: the bandwidth case
        case("attend-long", "attend", m7, seqs=4, rows=1, kv=131072, even=True, dtype="f16", fmt="int8"),
        # four drafted tokens of each sequence checked in one call
        case("attend-draft", "attend", m15, seqs=8, rows=4, kv=8000, even=False, dtype="f32", fmt="int8"),
        # a whole prompt attending to itself: the arithmetic case
        case("attend-prompt", "attend", m8, seqs=1, rows=8192, kv=8192, even=True, dtype="bf16", fmt="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice(HEADS)
    case = {"op": rng.choice(("rope", "write", "read", "attend", "attend")), "hq": hq, "hkv": hkv, "d": d,
            "dtype": rng.choice(tuple(TYPES))}
    if case["op"] == "rope":
        return {**case, "rows": _log(rng, 1, 8191 if case["dtype"] != "f32" else 4096), "norm": rng.random() < 0.7,
                "far": _log(rng, 16, 1 << 20)}
    case |= {"seqs": _log(rng, 1, 32), "even": rng.random() < 0.3, "fmt": rng.choice(tuple(FORMATS))}
    if case["op"] == "attend":
        most = 131072 * 4 * 4 // (case["seqs"] * hkv)  # the largest listed cache
        case["kv"] = _log(rng, 1, min(131072, most))
        # rows of a decode step, of a draft, or of a prompt; never more score entries than a listed case has
        room = (1 << 30) // (case["seqs"] * hq * case["kv"])
        case["rows"] = max(1, min(case["kv"], room, rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 8192)))))
    elif case["op"] == "write":
        case["rows"] = rng.choice((1, _log(rng, 2, 2 * 8000 // case["seqs"])))
        case["kv"] = case["rows"] + _log(rng, 1, 4096)
    else:
        case["rows"] = _log(rng, 1, 8 * 8000 // case["seqs"])
        case["kv"] = case["rows"] + rng.choice((0, _log(rng, 1, 2000)))
    return case


def _lengths(case):
    """(rows, kv) of every sequence, as lists, by the case alone: the longest has case['kv'], the others down to a
    hundredth of it."""
    n, rows, kv = case["seqs"], case["rows"], case["kv"]
    gen = torch.Generator().manual_seed(n + 100 * rows + 1000003 * kv)
    if case["even"] or n == 1:
        return [rows] * n, [kv] * n
    share = torch.rand(n, generator=gen).mul_(math.log(100)).neg_().exp_()
    share[int(torch.randint(n, (1,), generator=gen))] = 1.0
    kvs = [max(1, round(kv * float(s))) for s in share]
    if case["op"] == "read":
        return [max(0, min(k, round(rows * k / kv))) for k in kvs], kvs
    some = torch.randint(0, 2 * rows + 1, (n,), generator=gen).tolist() if rows > 8 else [rows] * n
    return [min(k, r) for k, r in zip(kvs, some)], kvs


def prepare(case, seed):
    dev, dt = "cuda", TYPES[case["dtype"]]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev).to(dtype)

    if case["op"] == "rope":
        n = case["rows"]
        s = {"qkv": normal(n, (hq + 2 * hkv) * d) * 3,  # rows of the fused projection: q, k, v side by side
             "pos": (torch.arange(n) + max(0, case["far"] - n)).to(torch.int32).to(dev),
             "q_out": torch.empty(n, hq, d, dtype=dt, device=dev), "k_out": torch.empty(n, hkv, d, dtype=dt, device=dev)}
        gains = [(1 + 0.2 * normal(d, dtype=torch.float32)).bfloat16() for _ in range(2)]
        s |= {"q_gain": gains[0], "k_gain": gains[1]} if case["norm"] else {"q_gain": None, "k_gain": None}
        s |= {"eps": 1e-6, "base": 1e6}
        return {"case": case, **s}

    rows, kvs = _lengths(case)
    n, pages = sum(rows), [-(-k // PAGE) for k in kvs]
    total, stride = sum(pages) + 3, max(pages)
    order = torch.randperm(total, generator=host).to(torch.int32)
    table = order[-1].repeat(case["seqs"], stride)  # entries behind a sequence's last page name a page of no sequence
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    # what earlier steps left in the cache: codes that reach the format's range, scales that differ by page and head
    codes = []
    for _ in range(2):
        x = torch.randn((total, hkv, PAGE, d), generator=gen, device=dev).mul_(CODE_MAX[case["fmt"]] / 3.5)
        x = x.clamp_(-CODE_MAX[case["fmt"]], CODE_MAX[case["fmt"]])
        codes.append(x.round_().to(torch.int8) if case["fmt"] == "int8" else x.to(torch.float8_e4m3fn))
    scales = [torch.rand((total, hkv), generator=gen, device=dev).add_(0.75).mul_(3.5 / CODE_MAX[case["fmt"]]) for _ in range(2)]
    starts = torch.zeros(case["seqs"] + 1, dtype=torch.int32)
    starts[1:] = torch.tensor(rows).cumsum(0)
    s = {"case": case, "k_codes": codes[0], "v_codes": codes[1], "k_scale": scales[0], "v_scale": scales[1],
         "table": table.to(dev), "row_start": starts.to(dev), "kv_len": torch.tensor(kvs, dtype=torch.int32).to(dev),
         "n": n, "most_rows": max(rows), "most_kv": max(kvs), "code_max": torch.tensor(CODE_MAX[case["fmt"]], device=dev)}
    if case["op"] == "write":
        kv = normal(n, 2, hkv, d)
        kv[:, 0, :, ::17] *= 4  # keys have channels that stand out
        s |= {"k": kv[:, 0], "v": kv[:, 1]}
    elif case["op"] == "read":
        s |= {"k_out": torch.empty(n, hkv, d, dtype=dt, device=dev), "v_out": torch.empty(n, hkv, d, dtype=dt, device=dev)}
    else:
        s |= {"q": normal(n, hq, d) * 2, "out": torch.empty(n, hq, d, dtype=dt, device=dev),
              "lse": torch.empty(n, hq, device=dev)}
    return s


# ---------------------------------------------------------------- the library's calls


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _handle(s):
    """The library and the cache's description (and the attention's workspace), which a program keeps."""
    if "handle" not in s:
        import ctypes

        import quantized_decode_gb300 as qd
        from quantized_decode_gb300 import _lib
        lib, c, cache = qd.load(), s["case"], None
        if c["op"] != "rope":
            cache = _lib.llm_kv8_cache(
                format=FORMATS[c["fmt"]], n_kv_heads=c["hkv"], head_dim=c["d"], n_pool_pages=s["k_codes"].shape[0],
                k_codes=s["k_codes"].data_ptr(), v_codes=s["v_codes"].data_ptr(), k_scale=s["k_scale"].data_ptr(),
                v_scale=s["v_scale"].data_ptr(), page_table=s["table"].data_ptr(), n_seqs=c["seqs"],
                table_stride=s["table"].shape[1])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if c["op"] == "attend":
            need = ctypes.c_int64()
            _lib.check(lib.llm_op_kv8_attention_workspace(ctypes.byref(cache), c["hq"], s["n"], ctypes.byref(need)),
                       "llm_op_kv8_attention_workspace")
            s["workspace"] = torch.zeros(need.value, dtype=torch.uint8, device="cuda")
        s["handle"] = lib, _lib.check, cache if cache is None else ctypes.byref(cache)
    return s["handle"]


def _own_rope(s):
    lib, check, _ = _handle(s)
    c, qkv = s["case"], s["qkv"]
    width, size = qkv.shape[1], qkv.element_size()
    gains = (s["q_gain"].data_ptr(), s["k_gain"].data_ptr()) if c["norm"] else (None, None)
    at = qkv.data_ptr()
    check(lib.llm_op_qk_norm_rope(TYPE_IDS[c["dtype"]], at, width, at + c["hq"] * c["d"] * size, width, *gains, s["eps"],
                                  s["base"], s["pos"].data_ptr(), c["rows"], c["hq"], c["hkv"], c["d"],
                                  s["q_out"].data_ptr(), s["k_out"].data_ptr(), _stream()), "llm_op_qk_norm_rope")
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_write(s):
    lib, check, cache = _handle(s)
    k, v = s["k"], s["v"]
    check(lib.llm_op_kv8_append(cache, TYPE_IDS[s["case"]["dtype"]], k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0),
                                s["row_start"].data_ptr(), s["kv_len"].data_ptr(), s["n"], s["err"].data_ptr(), _stream()),
          "llm_op_kv8_append")
    return {x: s[x] for x in ("k_codes", "v_codes", "k_scale", "v_scale")}


def _own_read(s):
    lib, check, cache = _handle(s)
    k, v = s["k_out"], s["v_out"]
    check(lib.llm_op_kv8_read(cache, TYPE_IDS[s["case"]["dtype"]], s["row_start"].data_ptr(), s["kv_len"].data_ptr(), s["n"],
                              k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), s["err"].data_ptr(), _stream()),
          "llm_op_kv8_read")
    return {"k": k, "v": v}


def _own_attend(s):
    lib, check, cache = _handle(s)
    q, w = s["q"], s["workspace"]
    check(lib.llm_op_kv8_attention(cache, TYPE_IDS[s["case"]["dtype"]], q.data_ptr(), q.stride(0), s["row_start"].data_ptr(),
                                   s["kv_len"].data_ptr(), s["n"], s["case"]["hq"], s["out"].data_ptr(), s["lse"].data_ptr(),
                                   w.data_ptr(), w.numel(), s["err"].data_ptr(), _stream()), "llm_op_kv8_attention")
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the plain forms


def _norm(x, gain, eps):
    return x if gain is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * gain.float()


def _plain_rope(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = s["qkv"].float().view(-1, hq + 2 * hkv, d)
    inv = torch.pow(torch.tensor(s["base"], dtype=torch.float64, device="cuda"),
                    torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / -d)
    angle = s["pos"].double()[:, None, None] * inv
    cos, sin = angle.cos().float(), angle.sin().float()

    def rotated(y, out):
        a, b = y[..., :d // 2], y[..., d // 2:]
        out.copy_(torch.cat((a * cos - b * sin, b * cos + a * sin), -1))
        return out

    return {"q": rotated(_norm(x[:, :hq], s["q_gain"], s["eps"]), s["q_out"]),
            "k": rotated(_norm(x[:, hq:hq + hkv], s["k_gain"], s["eps"]), s["k_out"])}


def _rows(s):
    """Of every row: its sequence, its position."""
    row = torch.arange(s["n"], device="cuda")
    start = s["row_start"].long()
    seq = torch.searchsorted(start[1:], row, right=True)
    return seq, s["kv_len"].long()[seq] - start[seq + 1] + row


def _coded(x, fmt, most):
    x = torch.maximum(torch.minimum(x, most), -most)
    return x.round().to(torch.int8) if fmt == "int8" else x.to(torch.float8_e4m3fn)


def _plain_write(s):
    fmt, most = s["case"]["fmt"], s["code_max"]
    seq, pos = _rows(s)
    table, start = s["table"].long(), s["row_start"].long()
    page, slot = table[seq, pos // PAGE], pos % PAGE
    # the page that each sequence's first row goes to, and how many tokens of it were there before
    count = start[1:] - start[:-1]
    first = s["kv_len"].long() - count
    here = (first % PAGE > 0) & (count > 0)
    begun = table.gather(1, (first // PAGE).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    earlier = torch.arange(PAGE, device="cuda")[None, :] < (first % PAGE)[:, None]

    def written(x, codes, scale):
        x, shape = x.float(), codes.shape
        bits = codes.view(torch.uint8)
        fresh = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]),
                                                        x.abs().amax(-1), "amax", include_self=True) / most
        old = scale[begun]
        grown = here[:, None] & (fresh[begun] > old)
        # a page that was begun keeps its scale unless the new rows need a larger one
        fresh[begun] = torch.where(here[:, None], torch.maximum(old, fresh[begun]), fresh[begun])
        ratio = torch.where(grown, old / fresh[begun], torch.ones_like(old))
        again = _coded(codes[begun].float() * ratio[..., None, None], fmt, most).view(torch.uint8)
        bits[begun] = torch.where(grown[..., None, None] & earlier[:, None, :, None], again, bits[begun])
        at = fresh[page][..., None]
        bits[page, :, slot] = _coded(torch.where(at > 0, x / at, torch.zeros_like(x)), fmt, most).view(torch.uint8)
        scale[page] = fresh[page]
        return bits.view(codes.dtype).view(shape)

    return {"k_codes": written(s["k"], s["k_codes"], s["k_scale"]), "v_codes": written(s["v"], s["v_codes"], s["v_scale"]),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_read(s):
    seq, pos = _rows(s)
    page, slot = s["table"].long()[seq, pos // PAGE], pos % PAGE

    def values(codes, scale, out):
        out.copy_(codes.view(torch.uint8)[page, :, slot].view(codes.dtype).float() * scale[page][..., None])
        return out

    return {"k": values(s["k_codes"], s["k_scale"], s["k_out"]), "v": values(s["v_codes"], s["v_scale"], s["v_out"])}


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d, b = c["hq"], c["hkv"], c["d"], c["seqs"]
    group, most, kv = hq // hkv, s["most_rows"], s["most_kv"]
    table = s["table"].long()

    def values(codes, scale):  # [sequence, kv head, token, d]
        x = codes.view(torch.uint8)[table].view(codes.dtype).float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(b, hkv, -1, d)[:, :, :kv]

    start, lens = s["row_start"].long(), s["kv_len"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(most, device="cuda")
    row = (start[:-1, None] + i).clamp(max=s["n"] - 1)
    q = s["q"][row].float().view(b, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * most, d)
    score = q @ values(s["k_codes"], s["k_scale"]).transpose(-1, -2)
    score = score.mul_(1 / math.sqrt(d)).view(b, hkv, group, most, kv)
    seen = torch.arange(kv, device="cuda") <= (lens - count)[:, None, None] + i[:, None]
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.view(b, hkv, group * most, kv) @ values(s["v_codes"], s["v_scale"])
    out = out.view(b, hkv, group, most, d) / torch.where(total > 0, total, torch.ones_like(total))
    seq, _ = _rows(s)
    at = torch.arange(s["n"], device="cuda") - start[seq]
    s["out"].copy_(out.permute(0, 3, 1, 2, 4)[seq, at].reshape(s["n"], hq, d))
    s["lse"].copy_((top + total.log())[..., 0].permute(0, 3, 1, 2)[seq, at].reshape(s["n"], hq))
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "write": _own_write, "read": _own_read, "attend": _own_attend}[op](state)
    return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        heads = case["rows"] * (hq + hkv)
        return {"bytes": heads * d * size * 2 + case["rows"] * 4, "flops": heads * d * (7 if case["norm"] else 3)}
    rows, kvs = _lengths(case)
    n, pages = sum(rows), sum(-(-k // PAGE) for k in kvs)
    if case["op"] == "attend":
        seen = sum(r * k - r * (r - 1) // 2 for r, k in zip(rows, kvs))
        return {"bytes": 2 * n * hq * d * size + n * hq * 4 + 2 * sum(kvs) * hkv * d + pages * (8 * hkv + 4),
                "flops": 4 * seen * hq * d}
    touched = sum(-(-k // PAGE) - (k - r) // PAGE for r, k in zip(rows, kvs) if r)
    return {"bytes": 2 * n * hkv * d * (size + 1) + touched * (8 * hkv + 4), "flops": 2 * n * hkv * d * (3 if case["op"] == "write" else 1)}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = s["qkv"].double().reshape(-1, hq + 2 * hkv, d)
    got = []
    for part, gain in ((x[:, :hq], s["q_gain"]), (x[:, hq:hq + hkv], s["k_gain"])):
        if gain is not None:
            part = part / (part.pow(2).sum(-1, keepdim=True) / d + s["eps"]).sqrt() * gain.double()
        turned = torch.empty_like(part)
        for i in range(d // 2):
            angle = s["pos"].double() * s["base"] ** (-2.0 * i / d)
            co, si = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            turned[..., i] = part[..., i] * co - part[..., i + d // 2] * si
            turned[..., i + d // 2] = part[..., i] * si + part[..., i + d // 2] * co
        got.append(turned)
    return {"q": got[0], "k": got[1]}


def _sequences(s):
    """(first row, rows, kv, pages) of each sequence."""
    start, kvs = s["row_start"].tolist(), s["kv_len"].tolist()
    for b, kv in enumerate(kvs):
        yield start[b], start[b + 1] - start[b], kv, s["table"][b, :-(-kv // PAGE)].long()


def _exact_write(s):
    """The scales alone: a code next to a half step may round either way."""
    got = {}
    for name, x in (("k", s["k"].double()), ("v", s["v"].double())):
        scale = s[name + "_scale"].double()
        for at, n, kv, pages in _sequences(s):
            if n == 0:
                continue
            first, last = (kv - n) // PAGE, (kv - 1) // PAGE
            largest = x[at:at + n].abs().amax(-1)
            slots = torch.zeros((last - first + 1) * PAGE, largest.shape[1], dtype=torch.float64, device="cuda")
            slots[(kv - n) % PAGE:(kv - n) % PAGE + n] = largest
            new = slots.view(-1, PAGE, largest.shape[1]).amax(1) / CODE_MAX[s["case"]["fmt"]]
            if (kv - n) % PAGE:
                new[0] = torch.maximum(new[0], scale[pages[first]])
            scale[pages[first:last + 1]] = new
        got[name + "_scale"] = scale
    return {"k_codes": None, "v_codes": None, **got}


def _exact_read(s):
    got = {}
    for name in ("k", "v"):
        parts = []
        for _, n, kv, pages in _sequences(s):
            x = s[name + "_codes"].view(torch.uint8)[pages].view(s[name + "_codes"].dtype).double()
            x = x * s[name + "_scale"][pages].double()[:, :, None, None]
            parts.append(x.permute(0, 2, 1, 3).flatten(0, 1)[kv - n:kv])
        got[name] = torch.cat(parts)
    return got


def _exact_attend(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if s["n"] * s["most_kv"] * hq * d > 1 << 42:
        return None
    out = torch.zeros(s["n"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["n"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for at, n, kv, pages in _sequences(s):
        if n == 0:
            continue
        hidden = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda")[:, None]
        for g in range(hkv):
            k, v = (s[x + "_codes"].view(torch.uint8)[pages, g].view(s["k_codes"].dtype).double()
                    * s[x + "_scale"][pages, g].double()[:, None, None] for x in ("k", "v"))
            k, v = k.reshape(-1, d)[:kv], v.reshape(-1, d)[:kv]
            for h in range(g * hq // hkv, (g + 1) * hq // hkv):
                w = s["q"][at:at + n, h].double() @ k.T / math.sqrt(d)
                w.masked_fill_(hidden, -math.inf)
                lse[at:at + n, h] = torch.logsumexp(w, -1)
                out[at:at + n, h] = torch.exp(w - lse[at:at + n, h, None]) @ v
    return {"out": out, "lse": lse}
