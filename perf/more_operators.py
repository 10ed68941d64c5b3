"""Cases, plain forms and 64-bit values of what stands before, between and after the halves of a decode step.

Four operators: the root-mean-square norm with the residual's addition
(``norm``), the projection with 8-bit weights of rows that are rounded to 8 bits
on the way, after that norm or as they are (``project``), the choice of the
best continuations over beams and vocabulary (``select``), and the reordering of
the paged cache by the beams that were chosen (``reorder``). ``run`` computes
them from elementary torch operations where ``own`` is false and through
``activation_sparse_ffn_gb300.sffn`` where it is true.

Rounding to 8 bits is defined by arithmetic in 32 bits, one rounding per
operation, so that the codes are defined: t = x + residual; f = 1 / sqrt(mean t^2
+ eps) in 64 bits, rounded once; y = (t f) weight; scale = max |y| / 127; code =
y / scale rounded to the nearest whole number.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F16_MAX = 65504.0
EPS = 1e-5
MOST_FLOPS = 2 * 4096 * 10240 * 8192      # of the largest listed product
MOST_LOGITS = 32 * 8 * 131072             # of the largest listed choice


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _norm(rows, width, dtype, residual=True, **kw):
    return dict(op="norm", rows=rows, width=width, dtype=dtype, residual=residual, **kw)


def _project(n, k, rows, dtype, norm, residual, **kw):
    return dict(op="project", n=n, k=k, rows=rows, dtype=dtype, norm=norm, residual=residual, **kw)


def _select(batch, beams, vocab, n_out, dtype, first=False, masked=0.0, done=0.0, **kw):
    return dict(op="select", batch=batch, beams=beams, vocab=vocab, n_out=n_out, dtype=dtype, first=first,
                masked=masked, done=done, **kw)


def _reorder(groups, beams, hkv, dim, group, page, length, ragged, dtype, **kw):
    return dict(op="reorder", groups=groups, beams=beams, hkv=hkv, dim=dim, group=group, page=page, length=length,
                ragged=ragged, dtype=dtype, **kw)


def listed():
    return [
        # between the halves of an 8192-wide layer, one token: the smallest call
        _norm(1, 8192, "f32", name="norm_d8192_b1"),
        # the same for the tokens of prompts
        _norm(8192, 8192, "bf16", name="norm_d8192_prompts"),
        # output projection of a 4096-wide layer for one token: rows as they are, the residual added to the product
        _project(4096, 4096, 1, "f32", False, True, name="project_d4096_b1"),
        # an odd number of outputs, an 11008-long contraction, five tokens
        _project(4099, 11008, 5, "f16", False, True, name="project_odd_b5"),
        # q, k and v projections (64 + 2 x 8 heads of 128) of an 8192-wide layer after its norm, 16 tokens
        _project(10240, 8192, 16, "bf16", True, False, name="project_qkv_d8192_b16"),
        # proposed tokens of 24 sequences checked together, 150 rows in all
        _project(10240, 8192, 150, "f16", True, False, name="project_qkv_d8192_b150"),
        # the same projections for the 4096 tokens of prompts
        _project(10240, 8192, 4096, "bf16", True, False, name="project_qkv_d8192_prompts"),
        # the first choice of a search with four beams, which start alike
        _select(1, 4, 32000, 8, "f32", first=True, name="select_b1_first"),
        # an odd vocabulary under a grammar that leaves a tenth of the tokens, a row that it leaves nothing, ended beams
        _select(7, 5, 50257, 10, "f16", masked=0.9, done=0.3, name="select_odd_masked"),
        # 32 searches of eight beams over a large vocabulary
        _select(32, 8, 131072, 16, "bf16", name="select_b32_v131072"),
        # one search with four beams
        _reorder(1, 4, 8, 128, 128, 16, 1000, False, "f32", name="reorder_b1"),
        # 64 searches of eight beams each, prompts of unequal lengths
        _reorder(64, 8, 8, 128, 128, 64, 4095, True, "bf16", name="reorder_b64_ragged"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "project", "project", "select", "select", "reorder"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op == "norm":
        width = _log(rng, 64, 16384)
        return _norm(_log(rng, 1, min(8192, (1 << 26) // width)), width, dtype, residual=rng.random() < 0.7)
    if op == "project":
        n, k = _log(rng, 64, 28672), 16 * _log(rng, 4, 1024)
        norm = rng.random() < 0.5
        return _project(n, k, _log(rng, 1, min(4096, MOST_FLOPS // (2 * n * k))), dtype, norm,
                        not norm and rng.random() < 0.7)
    if op == "select":
        beams, vocab = rng.choice((1, 2, 3, 4, 5, 8, 8, 16)), _log(rng, 1000, 262144)
        batch = _log(rng, 1, max(1, min(64, MOST_LOGITS // (beams * vocab))))
        return _select(batch, beams, vocab, beams * rng.choice((1, 2)), dtype, first=rng.random() < 0.2,
                       masked=rng.choice((0.0, 0.0, 0.5, 0.99)), done=rng.choice((0.0, 0.0, 0.3)))
    beams, dim = rng.choice((2, 3, 4, 5, 8, 16)), rng.choice((64, 128, 128, 256))
    hkv = rng.choice((1, 2, 4, 8, 8, 16))
    groups = _log(rng, 1, max(1, min(64, (1 << 28) // (beams * hkv * dim * 64))))
    return _reorder(groups, beams, hkv, dim, min(dim, rng.choice((32, 64, 128))), rng.choice((16, 32, 64)),
                    _log(rng, 1, 8192), rng.random() < 0.6, dtype)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, width, g):
    """Rows with a few channels an order of magnitude above the rest."""
    x = torch.randn(rows, width, generator=g, device="cuda")
    x[:, torch.randperm(width, generator=g, device="cuda")[: max(1, width // 512)]] *= 12.0
    return x


def _norm_inputs(case, seed):
    g, dtype = _gen(seed), DTYPES[case["dtype"]]
    x = _activations(case["rows"], case["width"], g).to(dtype)
    r = torch.randn(case["rows"], case["width"], generator=g, device="cuda").to(dtype) if case["residual"] else None
    return x, r, 1.0 + 0.2 * torch.randn(case["width"], generator=g, device="cuda")


def _project_inputs(case, seed):
    g, dtype, (n, k) = _gen(seed), DTYPES[case["dtype"]], (case["n"], case["k"])
    codes = torch.empty(n, k, dtype=torch.int8, device="cuda")
    for at in range(0, n, 4096):
        codes[at:at + 4096] = (32.0 * torch.randn(min(4096, n - at), k, generator=g, device="cuda")).round().clamp(-127, 127)
    scales = (0.75 + 0.5 * torch.rand(n, generator=g, device="cuda")) / (32.0 * math.sqrt(k))
    x = _activations(case["rows"], k, g).to(dtype)
    weight = 1.0 + 0.2 * torch.randn(k, generator=g, device="cuda") if case["norm"] else None
    r = torch.randn(case["rows"], n, generator=g, device="cuda").to(dtype) if case["residual"] else None
    return codes, scales, x, weight, r


def _select_inputs(case, seed):
    g, (batch, beams, vocab) = _gen(seed), (case["batch"], case["beams"], case["vocab"])
    logits = 2.5 * torch.randn(batch * beams, vocab, generator=g, device="cuda")
    if case["masked"]:
        logits[torch.rand(batch * beams, vocab, generator=g, device="cuda") < case["masked"]] = -math.inf
        logits[(batch * beams) // 2] = -math.inf                # nothing is left to this beam
    logits = logits.to(DTYPES[case["dtype"]])
    scores = -5.0 - 3.0 * torch.rand(batch, beams, generator=g, device="cuda")
    if case["first"]:
        scores = torch.full_like(scores, -math.inf)
        scores[:, 0] = 0.0
    done = torch.rand(batch, beams, generator=g, device="cuda") < case["done"] if case["done"] else None
    return logits, scores, done, vocab // 3                     # the last is the token that ends a sequence


def _lengths(case):
    """Cached tokens of each group of beams; the first has the case's own, ragged ones are spread below it."""
    part = [1.0 if i == 0 or not case["ragged"] else (0.6180339887498949 * i) % 1.0 for i in range(case["groups"])]
    return [max(1, int(case["length"] * f)) for f in part]


def _reorder_inputs(case, seed):
    """Two page tables, the tokens of every sequence's last page if it is not full, and the beams that go on."""
    g, dtype = _gen(seed), DTYPES[case["dtype"]]
    beams, page, lengths = case["beams"], case["page"], _lengths(case)
    n_seq, width = len(lengths) * beams, -(-case["length"] // page)
    s = {"n_pages": 2 * n_seq + 64, "dtype": dtype, "n_seq": n_seq}
    length = torch.tensor(lengths, device="cuda").repeat_interleave(beams)
    full, tail = length // page, length % page
    # pages below 64 are the full ones, which stay where they are; every sequence has a page of its own to write to in each table
    own_pages = 64 + torch.randperm(2 * n_seq, generator=g, device="cuda").view(2, n_seq)
    table = torch.randint(0, 64, (2, n_seq, width), generator=g, device="cuda")
    at = torch.arange(width, device="cuda")
    table = torch.where((at == full[:, None]) & (tail[:, None] > 0), own_pages[..., None], table)
    s["table"], s["table_out"] = table.to(torch.int32)
    s["kv_len"] = length.to(torch.int32)
    parent = torch.randint(0, beams, (len(lengths), beams), generator=g, device="cuda")
    s["parents"] = parent.to(torch.int32).flatten()
    s["start"] = torch.cat((tail.new_zeros(1), tail.cumsum(0))).to(torch.int32)
    s["tokens"] = beams * sum(n % page for n in lengths)
    s["k"] = torch.randn(s["tokens"], case["hkv"], case["dim"], generator=g, device="cuda").to(dtype)
    s["v"] = torch.randn(s["tokens"], case["hkv"], case["dim"], generator=g, device="cuda").to(dtype)
    return s


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "norm":
        s["x"], s["residual"], s["weight"] = _norm_inputs(case, seed)
        if own:
            s["y"], s["sum"] = torch.empty_like(s["x"]), torch.empty_like(s["x"]) if case["residual"] else None
    elif case["op"] == "project":
        codes, scales, s["x"], s["weight"], s["residual"] = _project_inputs(case, seed)
        if own:
            from activation_sparse_ffn_gb300 import sffn
            s["linear"] = sffn.Linear8.from_weights(codes, scales, max_batch=case["rows"])
            s["ws"] = s["linear"].workspace(case["rows"])
            s["rows8"] = torch.empty(case["rows"], case["k"], dtype=torch.int8, device="cuda")
            s["scales8"] = torch.empty(case["rows"], device="cuda")
            s["y"] = torch.empty(case["rows"], case["n"], dtype=s["x"].dtype, device="cuda")
        else:
            s |= {"codes": codes, "scales": scales}
    elif case["op"] == "select":
        s["logits"], s["scores"], s["done"], s["end"] = _select_inputs(case, seed)
        if own:
            from activation_sparse_ffn_gb300 import sffn
            batch, n_out = case["batch"], case["n_out"]
            s["beams"] = sffn.Beams(case["vocab"], case["beams"], n_out, max_batch=batch)
            s["ws"] = s["beams"].workspace(batch)
            s["out"] = torch.empty(batch, n_out, device="cuda")
            s["parents"], s["tokens"] = torch.empty(2, batch, n_out, dtype=torch.int32, device="cuda")
    else:
        s |= _reorder_inputs(case, seed)
        hkv, dim, group, page = case["hkv"], case["dim"], case["group"], case["page"]
        if own:
            from activation_sparse_ffn_gb300 import sffn
            s["cache"] = sffn.KvCache(s["n_pages"], page, hkv, dim, group)
            s["batch"] = sffn.KvBatch(s["table"], s["kv_len"])
            fill = sffn.KvBatch(s["table"], s["kv_len"], s["start"], s["tokens"])
            k, v = s.pop("k"), s.pop("v")
            sffn.sffn_kv_append(s["cache"].handle, fill, None, k, v, None, None)
            s["caches"] = sffn.KvCaches([s["cache"]])
            s["after"] = sffn.KvBatch(s["table_out"], s["kv_len"], s["start"], s["tokens"])
            s["k_out"], s["v_out"] = torch.empty_like(k), torch.empty_like(v)
        else:
            s["codes"] = torch.zeros(2, s["n_pages"] * page, hkv, dim // 2, dtype=torch.uint8, device="cuda")
            s["param"] = torch.zeros(2, s["n_pages"] * page, hkv, dim // group, 2, dtype=torch.float16, device="cuda")
            _, at = _tail(s, s["table"])
            _store(s, 0, at, s.pop("k").float(), group)
            _store(s, 1, at, s.pop("v").float(), group)
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _normed(x, residual, weight):
    """Rows in 32 bits after the residual's addition, and their norm."""
    t = x.float() if residual is None else x.float() + residual.float()
    f = (1.0 / torch.sqrt(t.double().square().mean(-1, keepdim=True) + EPS)).float()
    return t, (t * f) * weight


def _rounded(y):
    """Codes and scales of rows."""
    top = y.abs().amax(-1, keepdim=True)
    scale = torch.where(torch.isfinite(top), top / 127.0, math.nan)
    code = torch.round(y / scale).clamp(-127, 127)
    return torch.where(scale > 0, code, 0.0), scale


def _plain_norm(s):
    t, y = _normed(s["x"], s["residual"], s["weight"])
    return {"y": y.to(s["x"].dtype), "sum": None if s["residual"] is None else t.to(s["x"].dtype)}


def _plain_project(s):
    x = s["x"].float() if s["weight"] is None else _normed(s["x"], None, s["weight"])[1]
    code, scale = _rounded(x)
    y = (code @ s["codes"].float().T) * (scale * s["scales"])
    return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)


def _plain_select(s):
    case = s["case"]
    batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
    z = s["logits"].double()
    top = z.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(z - torch.where(torch.isinf(top), 0.0, top)).sum(-1, keepdim=True))
    z = torch.where(torch.isinf(lse), -math.inf, z - lse).view(batch, beams, vocab)     # an empty row has no candidates
    if s["done"] is not None:
        ends = torch.arange(vocab, device="cuda") == s["end"]
        z = torch.where(s["done"][..., None], torch.where(ends, 0.0, -math.inf), z)
    total = (z + s["scores"].double()[..., None]).flatten(1)
    best, place = torch.sort(total, descending=True, stable=True)
    best, place = best[:, :case["n_out"]], place[:, :case["n_out"]]
    place = torch.where(torch.isinf(best), 0, place)
    return {"scores": best.float(), "parents": (place // vocab).to(torch.int32),
            "tokens": (place % vocab).to(torch.int32)}


def _tail(s, table):
    """Sequence of each token of the pages that are not full, and its row in the cache by a page table."""
    page, start = s["case"]["page"], s["start"].long()
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(start[1:].contiguous(), row, right=True)
    length = s["kv_len"].long()[seq]
    return seq, table.long()[seq, length // page] * page + row - start[seq]


def _store(s, which, slot, x, group):
    """Rounds rows to 16 levels a group of channels and writes them to the cache rows `slot`."""
    x = x.unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    mid = (lo * 0.5 + hi * 0.5).clamp(-F16_MAX, F16_MAX).half()
    step = (torch.maximum(hi - mid.float(), mid.float() - lo) / 15.0).clamp(max=F16_MAX).half()
    u = torch.floor((x - mid.float()) * (1.0 / (2.0 * step.float())) + 8.0).clamp(0, 15)
    u = torch.where(step == 0, 8.0, u).to(torch.uint8).flatten(-2)
    s["codes"][which, slot] = u[..., 0::2] | (u[..., 1::2] << 4)
    s["param"][which, slot] = torch.cat((step, mid), -1)


def _values(codes, param):
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    u = u.unflatten(-1, (param.shape[-2], -1))
    return (param[..., 1:].float() + param[..., :1].float() * (2.0 * u - 15.0)).flatten(-2)


def _plain_reorder(s):
    case = s["case"]
    beams, page = case["beams"], case["page"]
    first = torch.arange(s["n_seq"], device="cuda") // beams * beams
    source = first + s["parents"].long()
    full = (s["kv_len"] // page)[:, None] > torch.arange(s["table"].shape[1], device="cuda")
    s["table_out"] = torch.where(full, s["table"][source], s["table_out"])
    seq, to = _tail(s, s["table_out"])
    at = torch.arange(s["tokens"], device="cuda") - s["start"].long()[seq]
    # every beam of a group has as many tokens in its last page
    rows = s["table"].long()[source[seq], s["kv_len"].long()[seq] // page] * page + at
    s["codes"][:, to] = s["codes"][:, rows]
    s["param"][:, to] = s["param"][:, rows]
    return {"table": s["table_out"], "k": _values(s["codes"][0, to], s["param"][0, to]).to(s["dtype"]),
            "v": _values(s["codes"][1, to], s["param"][1, to]).to(s["dtype"])}


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "project": _plain_project, "select": _plain_select,
                "reorder": _plain_reorder}[case["op"]](s)
    from activation_sparse_ffn_gb300 import sffn
    if case["op"] == "norm":
        sffn.sffn_norm(s["x"], s["weight"], EPS, s["residual"], s["sum"], s["y"])
        return {"y": s["y"], "sum": s["sum"]}
    if case["op"] == "project":
        if case["norm"]:
            sffn.sffn_norm(s["x"], s["weight"], EPS, codes=s["rows8"], scales=s["scales8"])
        else:
            sffn.sffn_quantize(s["x"], s["rows8"], s["scales8"])
        sffn.sffn_linear8_forward(s["linear"].handle, s["rows8"], s["scales8"], s["y"], s["residual"], s["ws"])
        return s["y"]
    if case["op"] == "select":
        sffn.sffn_beam_select(s["beams"].handle, s["logits"], s["scores"], s["out"], s["parents"], s["tokens"],
                              s["done"], s["end"], s["ws"])
        return {"scores": s["out"], "parents": s["parents"], "tokens": s["tokens"]}
    sffn.sffn_kv_reorder(s["caches"], s["batch"], s["parents"], case["beams"], s["table_out"])
    sffn.sffn_kv_gather(s["cache"].handle, s["after"], s["k_out"], s["v_out"])
    return {"table": s["table_out"], "k": s["k_out"], "v": s["v_out"]}


# --------------------------------------------------------------------------
# Work and 64-bit values
# --------------------------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        cells = case["rows"] * case["width"]
        return {"bytes": cells * e * (4 if case["residual"] else 2) + 4 * case["width"], "flops": 5 * cells}
    if case["op"] == "project":
        n, k, rows = case["n"], case["k"], case["rows"]
        moved = n * k + 4 * n + rows * k * e + rows * n * e * (2 if case["residual"] else 1) + (4 * k if case["norm"] else 0)
        return {"bytes": moved, "flops": 2 * rows * n * k}
    if case["op"] == "select":
        # beams that are not alive or have ended need none of their logits
        rows = case["batch"] * (1 if case["first"] else case["beams"]) * (1.0 - case["done"])
        cells = rows * case["vocab"]
        return {"bytes": cells * e + case["batch"] * (5 * case["beams"] + 12 * case["n_out"]), "flops": 4 * cells}
    tail = case["beams"] * sum(n % case["page"] for n in _lengths(case))
    table = case["beams"] * sum(n // case["page"] for n in _lengths(case))
    row = case["hkv"] * (case["dim"] + 8 * (case["dim"] // case["group"]))
    # the cached rows of the last pages read, written and read back, their values out, and the ids of the full pages
    return {"bytes": tail * (3 * row + 2 * case["hkv"] * case["dim"] * e) + 8 * table,
            "flops": 4 * tail * case["hkv"] * case["dim"]}


def _codes_of(x, weight):
    """The whole numbers and scales that rows are rounded to, which are given: arithmetic in 32 bits throughout."""
    if weight is not None:
        mean = torch.einsum("rk,rk->r", x.double(), x.double()) / x.shape[1]
        x = x.mul((mean + EPS).rsqrt().float()[:, None]).mul(weight)
    step = torch.linalg.vector_norm(x, math.inf, 1, True).div(127)
    return x.div(step).round().double(), step.double()


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
    if case["op"] == "norm":
        x, r, weight = _norm_inputs(case, seed)
        y, total = torch.empty(x.shape, dtype=torch.float64, device="cuda"), None
        total = None if r is None else torch.empty_like(y)
        for at in range(0, case["rows"], 1024):
            t = x[at:at + 1024].double()
            if r is not None:
                t = t.add(r[at:at + 1024].double())
                total[at:at + 1024] = t
            y[at:at + 1024] = t / (torch.einsum("rk,rk->r", t, t) / case["width"] + EPS).sqrt()[:, None] * weight.double()
        return {"y": y, "sum": total}
    if case["op"] == "project":
        codes, scales, x, weight, r = _project_inputs(case, seed)
        code, step = _codes_of(x.float(), weight)
        y = torch.empty(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        for at in range(0, case["n"], 1024):
            part = torch.einsum("rk,nk->rn", code, codes[at:at + 1024].double())
            y[:, at:at + 1024] = part * scales[at:at + 1024].double() * step
        return y if r is None else y + r.double()
    if case["op"] == "select":
        logits, scores, done, end = _select_inputs(case, seed)
        out = torch.full((case["batch"], case["n_out"]), -math.inf, dtype=torch.float64, device="cuda")
        parents, tokens = torch.zeros(2, *out.shape, dtype=torch.int32, device="cuda")
        for b in range(case["batch"]):
            found = []
            for j in range(case["beams"]):
                score = float(scores[b, j])
                if done is not None and bool(done[b, j]):
                    found.append((-score, j, end))
                    continue
                row = logits[b * case["beams"] + j].double().log_softmax(-1)
                if bool(row.isnan().any()) or math.isinf(score):
                    continue
                # the n_out best of a row, and whatever equals the last of them
                last = row.topk(min(case["n_out"], case["vocab"])).values[-1]
                at = torch.nonzero((row >= last) & (row > -math.inf))[:, 0]
                found += [(-(v + score), j, t) for v, t in zip(row[at].tolist(), at.tolist())]
            for i, (v, j, t) in enumerate(sorted(found)[:case["n_out"]]):
                out[b, i], parents[b, i], tokens[b, i] = -v, j, t
        return {"scores": out, "parents": parents, "tokens": tokens}
    s = _reorder_inputs(case, seed)
    table, start = s["table_out"].clone(), s["start"].tolist()
    source = [i // case["beams"] * case["beams"] + p for i, p in enumerate(s["parents"].tolist())]
    rows = torch.empty(s["tokens"], dtype=torch.long, device="cuda")
    for i, at in enumerate(source):
        n = int(s["kv_len"][i]) // case["page"]
        table[i, :n] = s["table"][at, :n]
        rows[start[i]:start[i + 1]] = torch.arange(start[at], start[at + 1], device="cuda")
    # what the cache holds is given: rounded to 16 levels in 32 bits
    return {"table": table, "k": _held(s["k"][rows].float(), case["group"]),
            "v": _held(s["v"][rows].float(), case["group"])}
