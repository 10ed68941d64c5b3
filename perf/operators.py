"""Cases, plain forms and 64-bit values of the attention half of a decode step.

Three operators around the sparse FFN layer: the projections with 4-bit weights
(``linear``), the append of a step's keys and values to a paged 4-bit cache with
the position rotation (``append``), and the attention over that cache
(``attend``). ``run`` computes them from elementary torch operations where
``own`` is false and through ``activation_sparse_ffn_gb300.sffn`` where it is
true.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F16_MAX = 65504.0


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _linear(n, k, group, batch, dtype, zeros=False, residual=False, **kw):
    return dict(op="linear", n=n, k=k, group=group, batch=batch, dtype=dtype, zeros=zeros, residual=residual, **kw)


def _cache(op, hq, hkv, dim, group, page, seqs, length, new, ragged, dtype, **kw):
    return dict(op=op, hq=hq, hkv=hkv, dim=dim, group=group, page=page, seqs=seqs, length=length, new=new,
                ragged=ragged, dtype=dtype, **kw)


def listed():
    return [
        # output projection of a 4096-wide layer for one token, with the residual: the smallest product
        _linear(4096, 4096, 128, 1, "f32", residual=True, name="linear_d4096_b1"),
        # q, k and v projections (64 + 2 x 8 heads of 128) of an 8192-wide layer for one token
        _linear(10240, 8192, 128, 1, "f32", name="linear_qkv_d8192_b1"),
        # an odd number of rows, an 11008-long contraction, groups of 32 with zero points, five tokens
        _linear(4099, 11008, 32, 5, "f16", zeros=True, name="linear_odd_zeros_b5"),
        # the 8192-wide projections for the largest batch of the library
        _linear(10240, 8192, 128, 32, "bf16", name="linear_qkv_d8192_b32"),
        # one token of one sequence, 8192-wide layer: latency
        _cache("append", 64, 8, 128, 128, 16, 1, 1000, 1, False, "f32", style="halves", rope=128, name="append_b1"),
        # one token each of 32 sequences, 128 heads of 64 over 8, half of the channels rotated in neighbouring pairs
        _cache("append", 128, 8, 64, 32, 32, 32, 4097, 1, True, "f16", style="pairs", rope=32, name="append_b32_d64"),
        # the prompts of five sequences of unequal lengths, 32 heads of 128 with their own keys
        _cache("append", 32, 32, 128, 64, 16, 5, 2500, 2500, True, "bf16", style="halves", rope=128,
               name="append_prompts"),
        # the start of a conversation: 33 cached tokens, one sequence
        _cache("attend", 64, 8, 128, 128, 16, 1, 33, 1, False, "f32", window=0, name="attend_b1_len33"),
        # one sequence with a long history
        _cache("attend", 64, 8, 128, 128, 64, 1, 131072, 1, False, "f32", window=0, name="attend_b1_len131072"),
        # 24 sequences of unequal lengths, 32 heads with their own keys, groups of 32
        _cache("attend", 32, 32, 128, 32, 16, 24, 4099, 1, True, "bf16", window=0, name="attend_b24_ragged"),
        # checking up to eight proposed tokens a sequence, 16 query heads a key head, sliding window
        _cache("attend", 128, 8, 64, 64, 32, 4, 8191, 8, True, "f16", window=4096, name="attend_verify_d64"),
        # the largest batch with long histories
        _cache("attend", 64, 8, 128, 128, 64, 32, 32768, 1, False, "bf16", window=0, name="attend_b32_len32768"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "append", "attend", "attend"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    group = rng.choice((32, 64, 128))
    if op == "linear":
        return _linear(_log(rng, 64, 11008), group * _log(rng, 4, 11008 // group), group, _log(rng, 1, 32), dtype,
                       zeros=rng.random() < 0.4, residual=rng.random() < 0.4)
    dim = rng.choice((64, 128, 128, 256))
    group = min(group, dim)
    hkv = rng.choice((1, 2, 4, 8, 8, 16, 32))
    hq = hkv * rng.choice((1, 2, 4, 5, 8, 16) if hkv <= 8 else (1, 2))
    page = rng.choice((16, 32, 64))
    ragged = rng.random() < 0.6
    if op == "append":
        length = _log(rng, 1, 8192)
        new = 1 if rng.random() < 0.5 else _log(rng, 1, length)
        seqs = _log(rng, 1, max(1, min(64, (1 << 27) // (new * (hq + 2 * hkv) * dim))))
        return _cache("append", hq, hkv, dim, group, page, seqs, length, new, ragged, dtype,
                      style=rng.choice(("halves", "pairs")), rope=rng.choice((0, dim // 2, dim)))
    length = _log(rng, 1, 131072)
    seqs = _log(rng, 1, max(1, min(64, (1 << 29) // (length * hkv * dim))))
    new = 1 if rng.random() < 0.6 else _log(rng, 1, min(32, max(1, (1 << 28) // (seqs * hq * length))))
    return _cache("attend", hq, hkv, dim, group, page, seqs, length, new, ragged, dtype,
                  window=0 if rng.random() < 0.7 else _log(rng, 1, 8192))


def _lengths(case):
    """(cached tokens, new tokens) of each sequence; the first has the case's own, ragged ones are spread below it."""
    part = [1.0 if i == 0 or not case["ragged"] else (0.6180339887498949 * i) % 1.0 for i in range(case["seqs"])]
    cached = [max(1, int(case["length"] * f)) for f in part]
    return [(n, min(n, max(1, int(case["new"] * f)))) for n, f in zip(cached, part)]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _linear_inputs(case, seed):
    g, (n, k) = _gen(seed), (case["n"], case["k"])
    codes = torch.randint(-8, 8, (n, k), generator=g, device="cuda", dtype=torch.int8)
    scales = (0.75 + 0.5 * torch.rand(n, k // case["group"], generator=g, device="cuda")) / (4.6 * math.sqrt(k))
    scales = scales.half()
    zeros = torch.randint(-3, 4, scales.shape, generator=g, device="cuda").half() if case["zeros"] else None
    x = torch.randn(case["batch"], k, generator=g, device="cuda")
    # a few channels an order of magnitude above the rest, as activations have them
    x[:, torch.randperm(k, generator=g, device="cuda")[: max(1, k // 512)]] *= 12.0
    dtype = DTYPES[case["dtype"]]
    r = torch.randn(case["batch"], n, generator=g, device="cuda").to(dtype) if case["residual"] else None
    return codes, scales, zeros, x.to(dtype), r


def _cache_inputs(case, seed):
    """Lengths, page table, the sequences' keys and values, and this step's rows."""
    g, dtype = _gen(seed), DTYPES[case["dtype"]]
    lengths = _lengths(case)
    hq, hkv, dim, page = case["hq"], case["hkv"], case["dim"], case["page"]
    total, fresh = sum(n for n, _ in lengths), sum(q for _, q in lengths)
    width = -(-case["length"] // page)
    n_pages = len(lengths) * width + 3
    table = torch.randperm(n_pages, generator=g, device="cuda")[: len(lengths) * width].view(len(lengths), width)
    s = {"table": table.to(torch.int32), "n_pages": n_pages, "dtype": dtype, "lengths": lengths}
    s["kv_len"] = torch.tensor([n for n, _ in lengths], dtype=torch.int32, device="cuda")
    counts = torch.tensor([0] + [q for _, q in lengths], device="cuda")
    s["q_start"] = counts.cumsum(0).to(torch.int32)
    s["fresh"] = fresh
    if case["op"] == "append":
        s["qkv"] = torch.randn(fresh, (hq + 2 * hkv) * dim, generator=g, device="cuda").to(dtype)
        if case["rope"]:
            # a model's table: base 10000, angles in 64 bits, rounded once
            j = torch.arange(case["rope"] // 2, device="cuda", dtype=torch.float64)
            angle = torch.arange(case["length"], device="cuda", dtype=torch.float64)[:, None] \
                * 10000.0 ** (-2.0 * j / case["rope"])
            s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()
        return s
    spread = 0.5 + 2.0 * torch.rand(hkv, dim, generator=g, device="cuda") ** 4   # some key channels stand out
    shift = torch.randn(hkv, dim, generator=g, device="cuda")
    s["k"] = (torch.randn(total, hkv, dim, generator=g, device="cuda") * spread + shift).to(dtype)
    s["v"] = torch.randn(total, hkv, dim, generator=g, device="cuda").to(dtype)
    s["q"] = torch.randn(fresh, hq, dim, generator=g, device="cuda").to(dtype)
    s["all_start"] = torch.tensor([0] + [n for n, _ in lengths], device="cuda").cumsum(0).to(torch.int32)
    s["total"] = total
    return s


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "linear":
        codes, scales, zeros, x, r = _linear_inputs(case, seed)
        s |= {"x": x, "residual": r}
        if own:
            from activation_sparse_ffn_gb300 import sffn
            s["linear"] = sffn.Linear.from_weights(codes, scales, zeros, max_batch=case["batch"])
            s["ws"] = s["linear"].workspace(case["batch"])
            s["y"] = torch.empty(case["batch"], case["n"], dtype=x.dtype, device="cuda")
        else:
            u = (codes + 8).to(torch.uint8)
            s |= {"packed": u[:, 0::2] | (u[:, 1::2] << 4), "scales": scales, "zeros": zeros}
        return s
    s |= _cache_inputs(case, seed)
    hq, hkv, dim, group, page = case["hq"], case["hkv"], case["dim"], case["group"], case["page"]
    if own:
        from activation_sparse_ffn_gb300 import sffn
        s["cache"] = sffn.KvCache(s["n_pages"], page, hkv, dim, group)
        s["batch"] = sffn.KvBatch(s["table"], s["kv_len"], s["q_start"], s["fresh"])
        if case["op"] == "append":
            s["rotation"] = sffn.Rope(s["rope"], case["style"]) if case["rope"] else None
            s["q_out"] = torch.empty(s["fresh"], hq, dim, dtype=s["dtype"], device="cuda")
            s["k_out"] = torch.empty(s["fresh"], hkv, dim, dtype=s["dtype"], device="cuda")
            s["v_out"] = torch.empty(s["fresh"], hkv, dim, dtype=s["dtype"], device="cuda")
        else:
            fill = sffn.KvBatch(s["table"], s["kv_len"], s.pop("all_start"), s.pop("total"))
            sffn.sffn_kv_append(s["cache"].handle, fill, None, s.pop("k"), s.pop("v"), None, None)
            s["ws"] = s["cache"].workspace(s["batch"], hq)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["fresh"], hq, device="cuda")
        return s
    s["codes"] = torch.zeros(2, s["n_pages"] * page, hkv, dim // 2, dtype=torch.uint8, device="cuda")
    s["param"] = torch.zeros(2, s["n_pages"] * page, hkv, dim // group, 2, dtype=torch.float16, device="cuda")
    if case["op"] == "attend":
        slot = _slots(s, s.pop("all_start"), s.pop("total"), page)[1]
        _store(s, 0, slot, s.pop("k").float(), group)
        _store(s, 1, slot, s.pop("v").float(), group)
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _slots(s, start, count, page):
    """Position and cache row of each of the last start[i + 1] - start[i] tokens of every sequence."""
    row = torch.arange(count, device="cuda")
    seq = torch.searchsorted(start[1:].long(), row, right=True)
    pos = s["kv_len"].long()[seq] - start.long()[seq + 1] + row
    return pos, s["table"].long()[seq, pos // page] * page + pos % page


def _store(s, which, slot, x, group):
    """Rounds rows to 16 levels a group of channels and writes them to the cache rows `slot`."""
    x = x.unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    mid = (lo * 0.5 + hi * 0.5).clamp(-F16_MAX, F16_MAX).half()
    far = torch.maximum(hi - mid.float(), mid.float() - lo)
    step = (far / 15.0).clamp(max=F16_MAX).half()
    inv = 1.0 / (2.0 * step.float())
    u = torch.floor((x - mid.float()) * inv + 8.0).clamp(0, 15)
    u = torch.where(step == 0, 8.0, u).to(torch.uint8).flatten(-2)
    s["codes"][which, slot] = u[..., 0::2] | (u[..., 1::2] << 4)
    s["param"][which, slot] = torch.cat((step, mid), -1)


def _values(codes, param):
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    u = u.unflatten(-1, (param.shape[-2], -1))
    return (param[..., 1:].float() + param[..., :1].float() * (2.0 * u - 15.0)).flatten(-2)


def _rotate(x, table, style):
    n = table.shape[-2]
    cos, sin, rest = table[:, None, :, 0], table[:, None, :, 1], x[..., 2 * n:]
    if style == "halves":
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
    a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)


def _plain_linear(s):
    p, group = s["packed"], s["case"]["group"]
    c = (torch.stack((p & 15, p >> 4), -1).flatten(-2).float() - 8.0).unflatten(-1, (-1, group))
    if s["zeros"] is not None:
        c = c - s["zeros"].float()[..., None]
    y = s["x"].float() @ (c * s["scales"].float()[..., None]).flatten(-2).T
    return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)


def _plain_append(s):
    case = s["case"]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    pos, slot = _slots(s, s["q_start"], s["fresh"], case["page"])
    q, k, v = s["qkv"].float().unflatten(-1, (-1, dim)).split((hq, hkv, hkv), 1)
    if case["rope"]:
        table = s["rope"][pos]
        q, k = _rotate(q, table, case["style"]), _rotate(k, table, case["style"])
    _store(s, 0, slot, k, case["group"])
    _store(s, 1, slot, v, case["group"])
    return {"q": q.to(s["dtype"]), "k": _values(s["codes"][0, slot], s["param"][0, slot]).to(s["dtype"]),
            "v": _values(s["codes"][1, slot], s["param"][1, slot]).to(s["dtype"])}


def _plain_attend(s):
    case = s["case"]
    hkv, dim, page, length = case["hkv"], case["dim"], case["page"], case["length"]
    at = torch.arange(length, device="cuda")
    rows = s["table"].long()[:, at // page] * page + at % page                       # (S, L)
    k = _values(s["codes"][0, rows], s["param"][0, rows]).transpose(1, 2)             # (S, Hkv, L, D)
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    i = torch.arange(case["new"], device="cuda")
    token = (start[:-1, None] + i).clamp(max=s["fresh"] - 1)                          # (S, Q), the rest is padding
    q = s["q"].float()[token].unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (q @ k.transpose(2, 3)) / math.sqrt(dim)
    del k
    pos = kv_len[:, None] - (start[1:] - start[:-1])[:, None] + i                     # (S, Q)
    seen = at <= pos[..., None]
    if case["window"]:
        seen = seen & (at > pos[..., None] - case["window"])
    seen = seen[:, None, :, None]                                                     # (S, 1, Q, 1, L)
    score = score.unflatten(2, (case["new"], -1)).masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    del score
    total = p.sum(-1, keepdim=True)
    v = _values(s["codes"][1, rows], s["param"][1, rows]).transpose(1, 2)
    o = (p.flatten(2, 3) @ v).unflatten(2, (case["new"], -1)) / torch.where(total == 0, 1.0, total)
    seq = torch.searchsorted(start[1:], torch.arange(s["fresh"], device="cuda"), right=True)
    nth = torch.arange(s["fresh"], device="cuda") - start[seq]
    pick = lambda t: t.permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, nth]                 # noqa: E731
    return {"out": pick(o).to(s["dtype"]), "lse": pick(top + torch.log(total))[..., 0]}


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"linear": _plain_linear, "append": _plain_append, "attend": _plain_attend}[case["op"]](s)
    from activation_sparse_ffn_gb300 import sffn
    if case["op"] == "linear":
        sffn.sffn_linear_forward(s["linear"].handle, s["x"], s["y"], s["residual"], s["ws"])
        return s["y"]
    if case["op"] == "append":
        q, k, v = s["qkv"].unflatten(-1, (-1, case["dim"])).split((case["hq"], case["hkv"], case["hkv"]), 1)
        sffn.sffn_kv_append(s["cache"].handle, s["batch"], q, k, v, s["q_out"], s["rotation"])
        sffn.sffn_kv_gather(s["cache"].handle, s["batch"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    sffn.sffn_attend(s["cache"].handle, s["batch"], s["q"], s["out"], s["lse"], 1.0 / math.sqrt(case["dim"]),
                     case["window"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------
# Work and 64-bit values
# --------------------------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "linear":
        n, k, b = case["n"], case["k"], case["batch"]
        per_group = 4 if case["zeros"] else 2
        moved = n * k / 2 + n * (k // case["group"]) * per_group + b * (k + n * (2 if case["residual"] else 1)) * e
        return {"bytes": moved, "flops": 2 * b * n * k}
    lengths, hq, hkv, dim = _lengths(case), case["hq"], case["hkv"], case["dim"]
    row = hkv * (dim + 8 * (dim // case["group"]))          # cached bytes of one token's keys and values
    if case["op"] == "append":
        fresh = sum(q for _, q in lengths)
        # rows in, rotated queries out, codes written and read back, their values out
        return {"bytes": fresh * ((2 * hq + 4 * hkv) * dim * e + 2 * row + 4 * case["rope"]),
                "flops": fresh * (3 * (hq + hkv) * case["rope"] + 12 * hkv * dim)}
    moved = flops = 0
    for n, new in lengths:
        w = case["window"] or n
        first = max(0, n - new - w + 1)
        moved += (n - first) * row + new * hq * (2 * dim * e + 4)
        flops += 4 * dim * hq * sum(min(w, n - new + i + 1) for i in range(new))
    return {"bytes": moved, "flops": flops}


def _held(x, group):
    """The values that rows of numbers have in the cache, in 64 bits, by arithmetic in the rows' own type."""
    shape, x = x.shape, x.reshape(-1, group)
    lo, hi = x.min(1).values, x.max(1).values
    mid = (lo / 2 + hi / 2).clamp(-F16_MAX, F16_MAX).half().to(x.dtype)
    step = (torch.maximum(hi - mid, mid - lo) / 15).clamp(max=F16_MAX).half().to(x.dtype)
    level = (x - mid[:, None]) * (1 / (2 * step[:, None])) + 8
    level = torch.where(step[:, None] > 0, level.floor().clamp(0, 15), torch.full_like(level, 8))
    return (mid.double()[:, None] + (2 * level.double() - 15) * step.double()[:, None]).reshape(shape)


def exact(case, seed):
    if case["op"] == "linear":
        codes, scales, zeros, x, r = _linear_inputs(case, seed)
        x, y = x.double(), torch.empty(case["batch"], case["n"], dtype=torch.float64, device="cuda")
        for at in range(0, case["n"], 512):
            w = codes[at:at + 512].double()
            if zeros is not None:
                w -= zeros[at:at + 512].double().repeat_interleave(case["group"], 1)
            w *= scales[at:at + 512].double().repeat_interleave(case["group"], 1)
            y[:, at:at + 512] = torch.einsum("bk,nk->bn", x, w)
        return y if r is None else y + r.double()
    s = _cache_inputs(case, seed)
    hq, hkv, dim, group = case["hq"], case["hkv"], case["dim"], case["group"]
    if case["op"] == "append":
        rows = s["qkv"].double().reshape(s["fresh"], -1, dim).clone()
        at = 0
        for n, new in s["lengths"] if case["rope"] else ():
            half, turn = case["rope"] // 2, s["rope"].double()[n - new:n, None]
            first = slice(0, half) if case["style"] == "halves" else slice(0, case["rope"], 2)
            second = slice(half, case["rope"]) if case["style"] == "halves" else slice(1, case["rope"], 2)
            part = rows[at:at + new, :hq + hkv]
            z = torch.complex(part[..., first], part[..., second]) * torch.complex(turn[..., 0], turn[..., 1])
            part[..., first], part[..., second] = z.real, z.imag
            at += new
        return {"q": rows[:, :hq], "k": _held(rows[:, hq:hq + hkv], group),
                "v": _held(rows[:, hq + hkv:], group)}
    out = torch.zeros(s["fresh"], hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["fresh"], hq, dtype=torch.float64, device="cuda")
    at = token = 0
    for n, new in s["lengths"]:
        # what the cache holds is given: rounded to 16 levels in 32 bits
        kv = [_held(t[at:at + n].float(), group) for t in (s["k"], s["v"])]
        for i in range(new):
            last = n - new + i + 1
            first = max(0, last - case["window"]) if case["window"] else 0
            q = s["q"][token].double().reshape(hkv, -1, dim)
            score = torch.einsum("hgd,lhd->hgl", q, kv[0][first:last]) * dim ** -0.5
            out[token] = torch.einsum("hgl,lhd->hgd", score.softmax(-1), kv[1][first:last]).reshape(hq, dim)
            lse[token] = score.logsumexp(-1).reshape(hq)
            token += 1
        at += n
    return {"out": out, "lse": lse}
