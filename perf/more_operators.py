"""What the 16-bit K/V cache operators are measured on: the q/k norm with a rotation over several axes that writes the
cache, attention of a batch whose sequences share prefixes, the weight that each cached token receives, and eviction by it.

Each case is one call of one operator (``op``):

  rope    RMS norm of every query and key head, rotation to a position on three axes, K and V into the pages
  attend  each sequence's last rows over the prefix that its group shares and causally over its own pages
  weigh   the attention weight that each of a sequence's cached tokens got from its last rows, summed up
  evict   the tokens of least weight taken out of the pages, each head's own, the others moved together

``run`` computes them in plain torch while ``own`` is false and calls the library's entry points
(include/llm_ops.h) while it is true.  Shapes: ``hq`` query and ``hkv`` key/value heads of ``d``, ``seqs``
sequences, ``rows`` new rows in each (spread around that number), ``kv`` tokens in the longest sequence with those rows
in it, ``groups`` shared prefixes of up to ``prefix`` tokens, ``pages`` the cache's type, ``dtype`` the rows'.
"""
import math

import torch

own = False

PAGE = 16
AXES = 3
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPE_IDS = {"f32": 0, "f16": 1, "bf16": 2}
HEADS = ((4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128))


def listed():
    def case(name, op, heads, **kw):
        hq, hkv, d = heads
        return {"name": name, "op": op, "hq": hq, "hkv": hkv, "d": d, **kw}

    tiny, m15, m7, m8 = HEADS
    return [
        # one decode step of eight sequences, fp32 rows as the engine's projections leave them: only latency counts
        case("rope-step", "rope", m8, seqs=8, rows=1, kv=4000, dtype="f32", pages="bf16", norm=True, mixed=False),
        # prompts of pictures and text, written at once
        case("rope-prompts", "rope", m7, seqs=4, rows=2000, kv=2000, dtype="bf16", pages="bf16", norm=False, mixed=True),
        # two short conversations behind a short system prompt on the smallest decoder: latency alone
        case("attend-pair", "attend", tiny, seqs=2, rows=1, kv=21, groups=1, prefix=301, pages="bf16"),
        # users of one assistant: a long prompt that all share, short conversations of their own
        case("attend-users", "attend", m8, seqs=32, rows=1, kv=500, groups=1, prefix=16384, pages="bf16"),
        # many samples of one prompt decoding together: the prefix alone is work for the tensor cores
        case("attend-crowd", "attend", m7, seqs=256, rows=1, kv=300, groups=1, prefix=8191, pages="f16"),
        # several assistants at once, each with its prompt and its users
        case("attend-groups", "attend", m8, seqs=64, rows=1, kv=1500, groups=4, prefix=12000, pages="bf16"),
        # five drafted tokens of each sequence checked behind a shared document
        case("attend-draft", "attend", m15, seqs=16, rows=5, kv=1000, groups=1, prefix=30011, pages="bf16"),
        # questions of 200 tokens about one document, taken in at once: the arithmetic case
        case("attend-questions", "attend", m8, seqs=8, rows=200, kv=200, groups=1, prefix=20000, pages="f16"),
        # the weights of a decode step of eight long conversations
        case("weigh-step", "weigh", m8, seqs=8, rows=1, kv=16000, pages="bf16"),
        # the weights of whole prompts, before the first eviction
        case("weigh-prompts", "weigh", m7, seqs=2, rows=4000, kv=4000, pages="f16"),
        # one conversation held to its budget, every 64 tokens
        case("evict-one", "evict", m15, seqs=1, kv=4159, budget=4096, first=4, last=512, pages="bf16"),
        # long prompts cut to a quarter after they were read
        case("evict-prompts", "evict", m8, seqs=16, kv=16384, budget=4096, first=4, last=1024, pages="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice(HEADS)
    case = {"op": rng.choice(("rope", "attend", "attend", "weigh", "evict")), "hq": hq, "hkv": hkv, "d": d,
            "pages": rng.choice(("f16", "bf16"))}
    if case["op"] == "rope":
        n = _log(rng, 1, 8000)
        case |= {"seqs": min(n, _log(rng, 1, 32)), "dtype": rng.choice(tuple(TYPES)), "norm": rng.random() < 0.5,
                 "mixed": rng.random() < 0.5}
        rows = max(1, n // case["seqs"])
        return {**case, "rows": rows, "kv": rows + rng.choice((0, _log(rng, 1, 4000)))}
    if case["op"] == "attend":
        case |= {"seqs": _log(rng, 1, 256), "prefix": _log(rng, 1, 32768)}
        case["groups"] = rng.choice((1, 1, min(case["seqs"], _log(rng, 1, 8))))
        # rows of a decode step, of a draft, or of a prompt; never more score entries or cache than a listed case has
        room = (1 << 29) // (case["seqs"] * hq * case["prefix"])
        case["kv"] = _log(rng, 1, min(8192, (1 << 17) * 8 // (case["seqs"] * hkv)))
        case["rows"] = max(1, min(case["kv"], room, rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 512)))))
        return case
    case["seqs"] = _log(rng, 1, 32)
    most = 16384 * 16 * 8 // (case["seqs"] * hkv) // 4
    case["kv"] = _log(rng, 1, min(65536, most))
    if case["op"] == "weigh":
        room = (1 << 29) // (case["seqs"] * hq * case["kv"])
        case["rows"] = max(1, min(case["kv"], room, rng.choice((1, 1, _log(rng, 2, 64), _log(rng, 65, 4000)))))
    else:
        case["budget"] = rng.choice((max(1, case["kv"] - _log(rng, 1, 64)), max(1, case["kv"] // _log(rng, 2, 16))))
        case["first"] = min(4, case["budget"] // 4)
        case["last"] = case["budget"] // rng.choice((2, 4, 8))
    return case


def _spread(case):
    """(rows, kv) of every sequence and the length of every prefix, as lists, by the case alone: the longest has
    case['kv'], the others down to a tenth of it."""
    n, rows, kv = case["seqs"], case.get("rows", 0), case["kv"]
    gen = torch.Generator().manual_seed(n + 100 * rows + 1000003 * kv)

    def lengths(count, most, least):
        share = torch.rand(count, generator=gen).mul_(math.log(least)).neg_().exp_()
        share[int(torch.randint(count, (1,), generator=gen))] = 1.0
        return [max(1, round(most * float(s))) for s in share]

    kvs = lengths(n, kv, 10)
    counts = [rows] * n
    if rows > 16:  # prompts differ, steps and drafts do not
        counts = [max(1, round(rows * f)) for f in (torch.rand(n, generator=gen) + 0.5).tolist()] if n > 1 else counts
        kvs = [max(k, r) for k, r in zip(kvs, counts)] if case["op"] != "rope" else kvs
    kvs = [max(k, r) for k, r in zip(kvs, counts)]
    return counts, kvs, lengths(case["groups"], case["prefix"], 4) if "groups" in case else []


def _axis_of(case):
    """The axis of each frequency: in sections one after another, or in turn."""
    half = case["d"] // 2
    if case["mixed"]:
        return [i % 3 if i < half * 15 // 16 else 0 for i in range(half)]
    return [0] * (half // 4) + [1] * (half * 3 // 8) + [2] * (half * 3 // 8)


def prepare(case, seed):
    dev, dt = "cuda", TYPES[case["pages"]]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["seqs"]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).to(dev)

    rows, kvs, prefixes = _spread(case)
    n, need = sum(rows), [-(-k // PAGE) for k in kvs + prefixes]
    total = sum(need) + 3
    order = torch.randperm(total, generator=host).to(torch.int32)
    tables, at = [], 0
    for lens in (need[:b], need[b:]):
        # entries behind a sequence's last page name a page of no sequence
        table = order[-1].repeat(len(lens), max(lens, default=1))
        for i, p in enumerate(lens):
            table[i, :p] = order[at:at + p]
            at += p
        tables.append(table.to(dev))
    starts = torch.zeros(b + 1, dtype=torch.int32)
    starts[1:] = torch.tensor(rows).cumsum(0)
    s = {"case": case, "k_pool": normal(total, hkv, PAGE, d), "v_pool": normal(total, hkv, PAGE, d), "table": tables[0],
         "kv_len": ints(kvs), "row_start": starts.to(dev), "n": n, "most_rows": max(rows), "most_kv": max(kvs)}
    if case["op"] == "rope":
        row = torch.arange(n)
        seq = torch.searchsorted(starts[1:].long(), row, right=True)
        token = torch.tensor(kvs)[seq] - starts[seq + 1] + row
        # every 1000 tokens 40 of text, which move on all axes alike, then a picture 32 wide that moves on its own two
        part, j = token // 1000 * 72, token % 1000
        inside = (j - 40).clamp(min=0)
        pos = torch.stack((part + j.clamp(max=40), part + j.clamp(max=40) + inside // 32, part + j.clamp(max=40) + inside % 32))
        s |= {"qkv": normal(n, (hq + 2 * hkv) * d, dtype=TYPES[case["dtype"]]) * 3,  # rows of the fused projection
              "pos": pos.to(torch.int32).to(dev), "axis": torch.tensor(_axis_of(case), dtype=torch.uint8),
              "q_out": torch.empty(n, hq, d, dtype=dt, device=dev), "eps": 1e-6, "base": 1e6}
        gains = [(1 + 0.2 * normal(d, dtype=torch.float32)).bfloat16() for _ in range(2)]
        return {**s, "q_gain": gains[0], "k_gain": gains[1]} if case["norm"] else {**s, "q_gain": None, "k_gain": None}
    if case["op"] == "evict":
        s |= {"scores": torch.rand(b, hkv, max(kvs) + 5, generator=gen, device=dev).pow_(-0.5).sub_(1.0),  # a few get most
              "scores_out": torch.zeros(b, hkv, max(kvs) + 5, device=dev),
              "kept": torch.full((b, hkv, case["budget"]), -1, dtype=torch.int32, device=dev),
              "new_len": torch.zeros(b, dtype=torch.int32, device=dev)}
        return s
    s |= {"q": normal(n, hq, d) * 2, "lse": torch.empty(n, hq, device=dev)}
    if case["op"] == "attend":
        cuts = [round(b * i / case["groups"]) for i in range(case["groups"] + 1)]
        s |= {"prefix_table": tables[1], "prefix_len": ints(prefixes), "seq_start": ints(cuts), "most_prefix": max(prefixes),
              "out": torch.empty(n, hq, d, dtype=dt, device=dev)}
    else:
        s["lse"].copy_(_log_sums(s))  # as the attention before it left them
        old = torch.rand(b, hkv, max(kvs) + 3, generator=gen, device=dev)
        s |= {"scores": old, "keep": 0.5}  # older rows count less and less
    return s


# ---------------------------------------------------------------- the library's calls


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _handle(s):
    """The library, the cache's description, the prefixes' and the attention's workspace, which a program keeps."""
    if "handle" not in s:
        import ctypes

        import quantized_decode_gb300 as qd
        from quantized_decode_gb300 import _lib
        lib, c, prefix = qd.load(), s["case"], None
        cache = ctypes.byref(_lib.llm_kv16_cache(
            dtype=TYPE_IDS[c["pages"]], n_kv_heads=c["hkv"], head_dim=c["d"], n_pool_pages=s["k_pool"].shape[0],
            k_pool=s["k_pool"].data_ptr(), v_pool=s["v_pool"].data_ptr(), page_table=s["table"].data_ptr(),
            n_seqs=c["seqs"], table_stride=s["table"].shape[1]))
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if c["op"] == "rope":
            s["axis_bytes"] = (ctypes.c_uint8 * (c["d"] // 2))(*s["axis"].tolist())
        if c["op"] == "attend":
            prefix = ctypes.byref(_lib.llm_kv16_prefix(
                page_table=s["prefix_table"].data_ptr(), len=s["prefix_len"].data_ptr(), seq_start=s["seq_start"].data_ptr(),
                n_groups=c["groups"], table_stride=s["prefix_table"].shape[1]))
            need = ctypes.c_int64()
            _lib.check(lib.llm_op_kv16_attention_workspace(cache, prefix, c["hq"], s["n"], ctypes.byref(need)),
                       "llm_op_kv16_attention_workspace")
            s["workspace"] = torch.zeros(need.value, dtype=torch.uint8, device="cuda")
        s["handle"] = lib, _lib.check, cache, prefix
    return s["handle"]


def _own_rope(s):
    lib, check, cache, _ = _handle(s)
    c, qkv = s["case"], s["qkv"]
    width, size = qkv.shape[1], qkv.element_size()
    at, k_at, v_at = (qkv.data_ptr() + h * c["d"] * size for h in (0, c["hq"], c["hq"] + c["hkv"]))
    gains = (s["q_gain"].data_ptr(), s["k_gain"].data_ptr()) if c["norm"] else (None, None)
    check(lib.llm_op_kv16_rope_append(cache, TYPE_IDS[c["dtype"]], at, width, k_at, width, v_at, width, *gains, s["eps"],
                                      s["base"], s["axis_bytes"], AXES, s["pos"].data_ptr(), s["row_start"].data_ptr(),
                                      s["kv_len"].data_ptr(), s["n"], c["hq"], s["q_out"].data_ptr(), s["err"].data_ptr(),
                                      _stream()), "llm_op_kv16_rope_append")
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _own_attend(s):
    lib, check, cache, prefix = _handle(s)
    q, w = s["q"], s["workspace"]
    check(lib.llm_op_kv16_attention(cache, prefix, q.data_ptr(), q.stride(0), s["row_start"].data_ptr(), s["kv_len"].data_ptr(),
                                    s["n"], s["case"]["hq"], s["out"].data_ptr(), s["lse"].data_ptr(), w.data_ptr(), w.numel(),
                                    s["err"].data_ptr(), _stream()), "llm_op_kv16_attention")
    return {"out": s["out"], "lse": s["lse"]}


def _own_weigh(s):
    lib, check, cache, _ = _handle(s)
    q, scores = s["q"], s["scores"]
    check(lib.llm_op_kv16_weigh(cache, q.data_ptr(), q.stride(0), s["row_start"].data_ptr(), s["kv_len"].data_ptr(), s["n"],
                                s["case"]["hq"], s["lse"].data_ptr(), s["keep"], scores.data_ptr(), scores.stride(1),
                                s["err"].data_ptr(), _stream()), "llm_op_kv16_weigh")
    return {"scores": scores}


def _own_evict(s):
    lib, check, cache, _ = _handle(s)
    c = s["case"]
    check(lib.llm_op_kv16_evict(cache, s["kv_len"].data_ptr(), c["budget"], c["first"], c["last"], s["scores"].data_ptr(),
                                s["scores_out"].data_ptr(), s["scores"].stride(1), s["kept"].data_ptr(), s["new_len"].data_ptr(),
                                s["err"].data_ptr(), _stream()), "llm_op_kv16_evict")
    return {x: s[x] for x in ("kept", "new_len", "scores_out", "k_pool", "v_pool")}


# ---------------------------------------------------------------- the plain forms


def _rows(s):
    """Of every row: its sequence, its slot."""
    row = torch.arange(s["n"], device="cuda")
    start = s["row_start"].long()
    seq = torch.searchsorted(start[1:], row, right=True)
    return seq, s["kv_len"].long()[seq] - start[seq + 1] + row


def _plain_rope(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = s["qkv"].float().view(-1, hq + 2 * hkv, d)
    inv = torch.pow(torch.tensor(s["base"], dtype=torch.float64, device="cuda"),
                    torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / -d)
    angle = s["pos"].double()[s["axis"].long().cuda()].T[:, None] * inv  # [row, 1, frequency], each on its axis
    cos, sin = angle.cos().float(), angle.sin().float()

    def rotated(y, gain):
        if gain is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * gain.float()
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    seq, pos = _rows(s)
    page, slot = s["table"].long()[seq, pos // PAGE], pos % PAGE
    s["q_out"].copy_(rotated(x[:, :hq], s["q_gain"]))
    s["k_pool"][page, :, slot] = rotated(x[:, hq:hq + hkv], s["k_gain"]).to(s["k_pool"].dtype)
    s["v_pool"][page, :, slot] = x[:, hq + hkv:].to(s["v_pool"].dtype)
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _part(q, table, k_pool, v_pool, seen):
    """Softmax statistics and weighted values of q [batch, rows, hq, d] over the pages of each batch entry; seen [batch,
    rows, tokens].  Without v_pool the scores alone."""
    n, most, hq, d = q.shape
    hkv, kv = k_pool.shape[1], seen.shape[-1]
    group = hq // hkv

    def values(pool):  # [batch, kv head, token, d]
        return pool[table.long()].float().transpose(1, 2).reshape(n, hkv, -1, d)[:, :, :kv]

    x = q.float().view(n, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * most, d)
    score = (x @ values(k_pool).transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(n, hkv, group, most, kv)
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    if v_pool is None:
        return score
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score.view(n, hkv, group * most, kv) @ values(v_pool)).view(n, hkv, group, most, d)
    return tuple(y.permute(0, 3, 1, 2, 4).reshape(n, most, hq, -1) for y in (top, total, out))


def _own_tokens(s, v_pool):
    """_part of each sequence's rows over its own tokens, [sequence, row], and where each row lies there."""
    start, lens, most = s["row_start"].long(), s["kv_len"].long(), s["most_rows"]
    count = start[1:] - start[:-1]
    i = torch.arange(most, device="cuda")
    row = (start[:-1, None] + i).clamp(max=s["n"] - 1)
    seen = torch.arange(s["most_kv"], device="cuda") <= (lens - count)[:, None, None] + i[:, None]
    seen &= (i < count[:, None])[..., None]
    seq, _ = _rows(s)
    return _part(s["q"][row], s["table"], s["k_pool"], v_pool, seen), (seq, torch.arange(s["n"], device="cuda") - start[seq])


def _log_sums(s):
    score, (seq, at) = _own_tokens(s, None)
    return torch.logsumexp(score, -1).permute(0, 3, 1, 2).reshape(*score.shape[:1], s["most_rows"], -1)[seq, at]


def _plain_attend(s):
    c, start, groups = s["case"], s["row_start"].long(), s["seq_start"].long()
    first = start[groups]  # the first row of each group
    count = first[1:] - first[:-1]
    # a group holds as many sequences as another, give or take one, but their rows differ: room for all rows where there are few
    most = s["n"] if c["groups"] == 1 else min(s["n"], (-(-c["seqs"] // c["groups"])) * s["most_rows"])
    i = torch.arange(most, device="cuda")
    row = (first[:-1, None] + i).clamp(max=s["n"] - 1)
    seen = torch.arange(s["most_prefix"], device="cuda") < s["prefix_len"].long()[:, None, None]
    prefix = _part(s["q"][row], s["prefix_table"], s["k_pool"], s["v_pool"], seen.expand(-1, most, -1))
    tail, where = _own_tokens(s, s["v_pool"])
    every = torch.arange(s["n"], device="cuda")
    group = torch.searchsorted(first[1:], every, right=True)
    parts = [x[group, every - first[group]] for x in prefix], [x[where] for x in tail]
    top = torch.maximum(parts[0][0], parts[1][0])
    factor = [torch.exp(p[0] - top) for p in parts]
    total = sum(p[1] * f for p, f in zip(parts, factor))
    s["out"].copy_(sum(p[2] * f for p, f in zip(parts, factor)) / total)
    s["lse"].copy_((top + total.log())[..., 0])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weigh(s):
    hkv, b, most, kv = s["case"]["hkv"], s["case"]["seqs"], s["most_rows"], s["most_kv"]
    score, (seq, at) = _own_tokens(s, None)
    lse = torch.zeros(b, most, hkv, score.shape[2], device="cuda")
    lse[seq, at] = s["lse"].view(s["n"], hkv, -1)
    got = score.sub_(lse.permute(0, 2, 3, 1)[..., None]).exp_().sum((2, 3))  # [sequence, kv head, token]
    token = torch.arange(kv, device="cuda")
    lens = s["kv_len"].long()
    first = lens - (s["row_start"][1:] - s["row_start"][:-1])
    now = s["scores"][..., :kv]
    new = torch.where((token < first[:, None])[:, None], s["keep"] * now, torch.zeros_like(now)) + got
    now.copy_(torch.where((token < lens[:, None])[:, None], new, now))
    return {"scores": s["scores"]}


def _plain_evict(s):
    c = s["case"]
    lens, kv, budget = s["kv_len"].long()[:, None, None], s["most_kv"], c["budget"]
    token = torch.arange(kv, device="cuda")
    score = s["scores"][..., :kv]
    rank = torch.where((token < c["first"]) | (token >= lens - c["last"]), torch.full_like(score, float("inf")), score)
    rank = torch.where(token < lens, rank, torch.full_like(score, float("-inf")))
    take = min(budget, kv)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :take]
    best = torch.where(torch.arange(take, device="cuda") < lens, best, torch.full_like(best, kv)).sort(-1).values
    there = best < kv
    at = best.clamp(max=kv - 1)
    seq = torch.arange(c["seqs"], device="cuda")[:, None, None].expand_as(at)
    head = torch.arange(c["hkv"], device="cuda")[None, :, None].expand_as(at)
    to = torch.arange(take, device="cuda").expand_as(at)
    table = s["table"].long()
    moves = there & (best != to)
    seq_m, head_m, from_m, to_m = seq[moves], head[moves], at[moves], to[moves]
    for x in ("k_pool", "v_pool"):
        rows = s[x][table[seq_m, from_m // PAGE], head_m, from_m % PAGE]
        s[x][table[seq_m, to_m // PAGE], head_m, to_m % PAGE] = rows
    s["kept"][..., :take] = torch.where(there, best, s["kept"][..., :take].long()).int()
    s["scores_out"][..., :take] = torch.where(there, score.gather(-1, at), s["scores_out"][..., :take])
    s["new_len"].copy_(s["kv_len"].clamp(max=budget))
    return {x: s[x] for x in ("kept", "new_len", "scores_out", "k_pool", "v_pool")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attend": _own_attend, "weigh": _own_weigh, "evict": _own_evict}[op](state)
    return {"rope": _plain_rope, "attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows, kvs, prefixes = _spread(case)
    n, pages = sum(rows), sum(-(-k // PAGE) for k in kvs + prefixes)
    seen = sum(r * k - r * (r - 1) // 2 for r, k in zip(rows, kvs))
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        touched = sum(-(-k // PAGE) - (k - r) // PAGE for r, k in zip(rows, kvs))
        return {"bytes": n * (hq + 2 * hkv) * d * (size + 2) + n * AXES * 4 + touched * 4,
                "flops": n * (hq + hkv) * d * (7 if case["norm"] else 3)}
    if case["op"] == "attend":
        b, groups = case["seqs"], case["groups"]
        for g, p in enumerate(prefixes):
            seen += p * sum(rows[round(b * g / groups):round(b * (g + 1) / groups)])
        return {"bytes": 4 * n * hq * d + n * hq * 4 + 4 * sum(kvs + prefixes) * hkv * d + pages * 4, "flops": 4 * seen * hq * d}
    if case["op"] == "weigh":
        return {"bytes": 2 * n * hq * d + n * hq * 4 + sum(kvs) * hkv * (2 * d + 8) + pages * 4, "flops": 2 * seen * hq * d}
    # every score is read; of the kept tokens those behind the first that goes are moved, all but a few
    kept = sum(min(k, case["budget"]) for k in kvs)
    moved = sum(min(k, case["budget"]) - case["first"] for k in kvs if k > case["budget"])
    return {"bytes": hkv * (sum(kvs) * 4 + kept * 8 + max(0, moved) * 2 * 2 * 2 * d) + pages * 4, "flops": sum(kvs) * hkv}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _sequences(s):
    """(first row, rows, kv, slots) of each sequence; slots: where its tokens lie in a pool seen as [page, token]."""
    start, kvs = s["row_start"].tolist(), s["kv_len"].tolist()
    for b, kv in enumerate(kvs):
        yield start[b], start[b + 1] - start[b], kv, _slots(s["table"][b], kv)


def _slots(pages, kv):
    t = torch.arange(kv, device="cuda")
    return pages.long()[t // PAGE], t % PAGE


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
            angle = s["pos"][int(s["axis"][i])].double() * s["base"] ** (-2.0 * i / d)
            co, si = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            turned[..., i] = part[..., i] * co - part[..., i + d // 2] * si
            turned[..., i + d // 2] = part[..., i] * si + part[..., i + d // 2] * co
        got.append(turned)
    pools = {"k": s["k_pool"].double(), "v": s["v_pool"].double()}
    for at, n, kv, (page, slot) in _sequences(s):
        pools["k"][page[kv - n:], :, slot[kv - n:]] = got[1][at:at + n]
        pools["v"][page[kv - n:], :, slot[kv - n:]] = x[at:at + n, hq + hkv:]
    return {"q": got[0], **pools}


def _exact_attend(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    out = torch.zeros(s["n"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["n"], hq), -math.inf, dtype=torch.float64, device="cuda")
    cuts = s["seq_start"].tolist()
    for b, (at, n, kv, (page, slot)) in enumerate(_sequences(s)):
        g = next(g for g in range(c["groups"]) if b < cuts[g + 1])
        before, before_slot = _slots(s["prefix_table"][g], int(s["prefix_len"][g]))
        page, slot, p = torch.cat((before, page)), torch.cat((before_slot, slot)), len(before)
        last = p + torch.arange(kv - n, kv, device="cuda")
        hidden = torch.arange(p + kv, device="cuda")[None, :] > last[:, None]
        k, v = s["k_pool"][page, :, slot].double(), s["v_pool"][page, :, slot].double()
        for h in range(hkv):
            for i in range(h * hq // hkv, (h + 1) * hq // hkv):
                w = (s["q"][at:at + n, i].double() @ k[:, h].T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                lse[at:at + n, i] = torch.logsumexp(w, -1)
                out[at:at + n, i] = torch.exp(w - lse[at:at + n, i, None]) @ v[:, h]
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    hq, hkv, d = (s["case"][x] for x in ("hq", "hkv", "d"))
    scores = s["scores"].double()
    for b, (at, n, kv, (page, slot)) in enumerate(_sequences(s)):
        hidden = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda")[:, None]
        scores[b, :, kv - n:kv] = 0
        scores[b, :, :kv] *= s["keep"]
        k = s["k_pool"][page, :, slot].double()
        for i in range(hq):
            w = s["q"][at:at + n, i].double() @ k[:, i * hkv // hq].T / math.sqrt(d) - s["lse"][at:at + n, i, None].double()
            scores[b, i * hkv // hq, :kv] += torch.exp(w).masked_fill_(hidden, 0.0).sum(0)
    return {"scores": scores}


def _exact_evict(s):
    """The scores alone: everything else is whole numbers or a copy."""
    c, scores = s["case"], s["scores_out"].double()
    for b, kv in enumerate(s["kv_len"].tolist()):
        for h in range(c["hkv"]):
            x = s["scores"][b, h, :kv].double()
            if kv > c["budget"]:
                middle = x[c["first"]:kv - c["last"]]
                order = torch.topk(middle, c["budget"] - c["first"] - c["last"]).indices.sort().values
                x = torch.cat((x[:c["first"]], middle[order], x[kv - c["last"]:]))
            scores[b, h, :len(x)] = x
    return {"kept": None, "new_len": None, "scores_out": scores, "k_pool": None, "v_pool": None}
