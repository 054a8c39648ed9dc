"""More operators of a served batch, as they are measured: cases, inputs, plain forms and 64-bit values.

A decode step over a cache that holds Q8_0 blocks (32 int8 codes and one f16 scale), down to the token:

  store      bias, QK-norm and rotary positions of the fused Q|K|V rows; K and V quantized into their slots
  read       rows of the cache read back as floats, as a prompt's next chunk needs them
  attention  one new token per request over its quantized pages
  sample     the next token from logits rows: top-k, top-p, min-p, temperature, from given random numbers

Head layouts (query heads / KV heads / head dim) and vocabularies are those of the configurations in synth/.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
HEADS = [(4, 2, 64), (14, 2, 64), (12, 2, 128), (28, 4, 128), (16, 8, 128)]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decode step of a batch, fused Q|K|V rows straight from a 16-bit projection (latency)
        dict(name="store decode 64", op="store", rows=64, nh=14, nkv=2, hd=64, src="bf16", to="bf16", page=16, style="half", rot=64, scaling="none",
             norm=False, bias=True, first=700, pad=0, order="rows"),
        # a long prompt chunk of the widest layout, f32 sums of the quantized GEMM, positions past the trained context
        dict(name="store prefill 4096 yarn", op="store", rows=4096, nh=28, nkv=4, hd=128, src="f32", to="bf16", page=16, style="half", rot=128,
             scaling="yarn", norm=False, bias=True, first=60000, pad=0, order="heads"),
        # a ragged chunk with QK-norm, half of each head rotated in interleaved pairs, padding rows at the end of a captured step
        dict(name="store norm 1001", op="store", rows=1001, nh=16, nkv=8, hd=128, src="f16", to="f16", page=32, style="interleaved", rot=64,
             scaling="linear", norm=True, bias=False, first=3, pad=23, order="heads"),
        # one short prompt's rows for its next chunk, into f32 regions (latency)
        dict(name="read 513", op="read", rows=513, nkv=2, hd=64, type="f32", page=16, order="rows"),
        # the rows of a batch whose pages move to 16-bit ones
        dict(name="read 131071", op="read", rows=131071, nkv=4, hd=128, type="bf16", page=64, order="heads"),
        # one request after a 512-token prompt (latency, split over the length)
        dict(name="attention 1 x 513", op="attention", n=1, lens="same", max_len=513, nh=14, nkv=2, hd=64, type="bf16", page=16, order="rows"),
        # a full serving batch, lengths spread up to 4096, one empty request
        dict(name="attention 64 x 4096", op="attention", n=64, lens="ragged", max_len=4096, nh=28, nkv=4, hd=128, type="bf16", page=16, order="heads"),
        # one very long context
        dict(name="attention 1 x 131071", op="attention", n=1, lens="same", max_len=131071, nh=12, nkv=2, hd=128, type="f16", page=64, order="heads"),
        # f32 queries, as the framework's own forward has them
        dict(name="attention 33 x 2048 f32", op="attention", n=33, lens="ragged", max_len=2048, nh=14, nkv=2, hd=64, type="f32", page=32, order="rows"),
        # the token of one decode step (latency)
        dict(name="sample 1 x 151936", op="sample", rows=1, vocab=151936, type="f32", mix="k and p", first=False, masked=False, extra=0),
        # a large batch whose requests all bring settings of their own: greedy, unfiltered, top-k, top-p, min-p and several at once
        dict(name="sample 512 x 151936", op="sample", rows=512, vocab=151936, type="f32", mix="mixed", first=False, masked=False, extra=0),
        # 16-bit logits under a grammar mask, nucleus alone, odd vocabulary and row stride, one row with nothing left
        dict(name="sample 65 x 150001", op="sample", rows=65, vocab=150001, type="bf16", mix="p", first=True, masked=True, extra=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "store", "read", "attention", "attention", "attention", "sample", "sample", "sample"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    nh, nkv, hd = rng.choice(HEADS)
    order = rng.choice(["rows", "heads"])
    if op == "store":
        src, to = rng.choice([("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
        norm = rng.random() < 0.4
        rows = _log(rng, 1, 2048 if src == "f32" else 4096)
        return dict(op=op, rows=rows, nh=nh, nkv=nkv, hd=hd, src=src, to=to, page=page, style=rng.choice(["half", "interleaved"]),
                    rot=rng.choice([hd, hd, hd // 2, hd // 4, 24]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]), norm=norm,
                    bias=not norm, first=_log(rng, 1, 1000000), pad=rng.choice([0, 0, rng.randrange(0, rows)]), order=order)
    if op == "read":
        t = rng.choice(["f32", "f16", "bf16"])
        return dict(op=op, rows=_log(rng, 1, 131071 * 4 * 128 * 2 // (nkv * hd * SIZE[t])), nkv=nkv, hd=hd, type=t, page=page, order=order)
    if op == "attention":
        t = rng.choice(["f32", "f16", "bf16", "bf16"])
        length = _log(rng, 1, 100000)
        most = max(1, min(256, 64 * 4096 * 4 * 128 // (length * nkv * hd)))
        return dict(op=op, n=_log(rng, 1, most), lens=rng.choice(["same", "ragged", "ragged"]), max_len=length, nh=nh, nkv=nkv, hd=hd, type=t,
                    page=page, order=order)
    vocab = rng.choice([4096, 151936, 152064, _log(rng, 33, 152064)])
    return dict(op=op, rows=_log(rng, 1, min(512, 256 * 151936 // vocab)), vocab=vocab, type=rng.choice(["f32", "f32", "f16", "bf16"]),
                mix=rng.choice(["greedy", "plain", "k", "k and p", "k and p", "p", "min", "mixed", "mixed"]), first=rng.random() < 0.5,
                masked=rng.random() < 0.4, extra=rng.choice([0, 0, 1, 7, 64]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(g, n_pages, page, nkv, hd, order, sigma):
    """Codes and scales [n_pages, page, nkv, ...] of normal rows: the rows of all heads behind one another, or each head's rows of a page."""
    shape = (n_pages, page, nkv) if order == "rows" else (n_pages, nkv, page)
    turn = (0, 1, 2, 3) if order == "rows" else (0, 2, 1, 3)
    codes = torch.empty(*shape, hd, dtype=torch.int8, device="cuda")
    scales = torch.empty(*shape, hd // 32, dtype=torch.float16, device="cuda")
    for c, s in zip(codes.split(4096), scales.split(4096)):
        x = sigma * torch.randn(*c.shape[:-1], hd // 32, 32, generator=g, device="cuda")
        d = x.abs().amax(-1, keepdim=True) / 127
        c.copy_(torch.round(x / d).to(torch.int8).flatten(-2))
        s.copy_(d[..., 0])
    return codes.permute(turn), scales.permute(turn)


def _cache(s, case, g, n_pages, sigma=1.0):
    s["k"], s["ks"] = _pool(g, n_pages, case["page"], case["nkv"], case["hd"], case["order"], sigma)
    s["v"], s["vs"] = _pool(g, n_pages, case["page"], case["nkv"], case["hd"], case["order"], sigma)
    if own:
        import quantized_transformer_prefill_gb300 as qp
        s["cache"] = qp.PagedCacheQ8(s["k"], s["v"], s["ks"], s["vs"])


def _rope_args(case):
    kind = case["scaling"]
    return dict(rot_dim=case["rot"], theta=1.0e6, style=case["style"], scaling=kind, factor=1.0 if kind == "none" else 4.0,
                n_ctx_orig=32768 if kind == "yarn" else 0)


def _prepare_store(case, g):
    rows, nh, nkv, hd, P = case["rows"], case["nh"], case["nkv"], case["hd"], case["page"]
    width = (nh + 2 * nkv) * hd
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n_pages = -(-rows // P) + 3
    pos = torch.arange(rows, device="cuda", dtype=torch.int32) + case["first"]
    slot = torch.randperm(n_pages * P, generator=g, device="cuda")[:rows].to(torch.int32)
    live = rows - case["pad"]
    pos[live:] = -1
    slot[live:] = -1
    # the whole pool is read back after the step, as 16-bit values
    back = lambda: torch.empty(n_pages * P, nkv * hd, dtype=torch.float16, device="cuda")  # noqa: E731
    s = dict(qkv=(1.5 * new(rows, width)).to(TYPES[case["src"]]), pos=pos, slot=slot, bias=None, q_norm=None, k_norm=None,
             out=torch.zeros(rows, nh * hd, dtype=TYPES[case["to"]], device="cuda"), back=(back(), back()),
             every=torch.arange(n_pages * P, dtype=torch.int32, device="cuda"))
    _cache(s, case, g, n_pages)
    if case["bias"]:
        s["bias"] = 0.5 * new(width)
    if case["norm"]:
        s["q_norm"], s["k_norm"] = 1 + 0.1 * new(hd), 1 + 0.1 * new(hd)
    if own:
        import quantized_transformer_prefill_gb300 as qp
        s["rope"] = qp.RopeTable(hd, **_rope_args(case))
    return s


def _prepare_read(case, g):
    rows, nkv, hd, P = case["rows"], case["nkv"], case["hd"], case["page"]
    n_pages = -(-rows // P) + 3
    # the rows of pages in an order of their own, page by page, as tables have them
    slot = (torch.randperm(n_pages, generator=g, device="cuda")[:, None] * P + torch.arange(P, device="cuda")).flatten()[:rows].to(torch.int32)
    out = lambda: torch.empty(rows, nkv * hd, dtype=TYPES[case["type"]], device="cuda")  # noqa: E731
    s = dict(slot=slot, out=(out(), out()))
    _cache(s, case, g, n_pages)
    return s


def _prepare_attention(case, g):
    n, nh, hd, P = case["n"], case["nh"], case["hd"], case["page"]
    t, W = TYPES[case["type"]], -(-case["max_len"] // P)
    length = torch.full((n,), case["max_len"], dtype=torch.int32, device="cuda")
    if case["lens"] == "ragged":
        length = torch.randint(1, case["max_len"] + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        length[n // 2] = 0
        length[0] = case["max_len"]
    held = -(-length.long() // P)
    n_pages = int(held.sum()) + 2
    table = torch.full((n, W), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(W, device="cuda")[None, :] < held[:, None]] = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)[:n_pages - 2]
    s = dict(q=(1.3 * torch.randn(n, nh * hd, generator=g, device="cuda")).to(t), table=table, length=length,
             out=torch.empty(n, nh * hd, dtype=t, device="cuda"), lse=torch.empty(n, nh, device="cuda"))
    _cache(s, case, g, n_pages)
    if own:
        import quantized_transformer_prefill_gb300 as qp
        s["work"] = qp.op_paged_attention_q8_workspace(s["cache"], n, nh)
    return s


def _prepare_sample(case, g):
    rows, V, t, mix = case["rows"], case["vocab"], TYPES[case["type"]], case["mix"]
    x = torch.empty(rows, V + case["extra"], device="cuda", dtype=t)
    x.normal_(0.0, 2.5, generator=g)
    # a few likely tokens above the rest, as a trained model's head gives them
    likely = (torch.randint(0, V, (rows, 1), generator=g, device="cuda") + torch.arange(6, device="cuda") * max(1, V // 7)) % V
    x.scatter_(1, likely, (16 + 2 * torch.randn(rows, 6, generator=g, device="cuda")).to(t))
    if case["masked"]:
        x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < 0.5, -math.inf)
        x[rows // 2].fill_(-math.inf)
    rand = lambda: torch.rand(rows, generator=g, device="cuda")  # noqa: E731
    # what each request asks for: 0 greedy, 1 no filter, 2 top-k, 3 top-k and top-p, 4 top-p, 5 min-p, 6 all of them
    what = torch.randint(0, 7, (rows,), generator=g, device="cuda")
    if mix != "mixed":
        what = torch.full((rows,), {"greedy": 0, "plain": 1, "k": 2, "k and p": 3, "p": 4, "min": 5}[mix], device="cuda")
    has = lambda *kinds: sum(what == k for k in kinds).bool()  # noqa: E731
    k = torch.tensor([1, 5, 20, 40, 50, 100, 1000, V], device="cuda")[torch.randint(0, 8, (rows,), generator=g, device="cuda")].clamp(max=V)
    return dict(x=x[:, :V], u=rand(), temperature=torch.where(has(0), 0.0, 0.5 + 0.8 * rand()), top_k=torch.where(has(2, 3, 6), k, 0).to(torch.int32),
                top_p=torch.where(has(3, 4, 6), 0.5 + 0.49 * rand(), 1.0), min_p=torch.where(has(5, 6), 0.01 + 0.1 * rand(), 0.0),
                out=(torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")))


def prepare(case, seed):
    s = {"store": _prepare_store, "read": _prepare_read, "attention": _prepare_attention, "sample": _prepare_sample}[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _values(codes, scales):
    """The values that Q8_0 blocks stand for."""
    return (codes.float().unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _frequencies(case, device):
    """Radians a position of each pair, and the factor on cos and sin, in 64 bits."""
    a, rot = _rope_args(case), case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    theta, s, scale = a["theta"], a["factor"], 1.0
    if a["scaling"] == "ntk" and rot > 2:
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if a["scaling"] == "linear":
        f = f / s
    if a["scaling"] == "yarn":
        dim = lambda turns: rot * math.log(a["n_ctx_orig"] / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / s * ramp + f * (1 - ramp)
        scale = 0.1 * math.log(s) + 1
    return f, scale


def _turn(x, cos, sin, case):
    """Pairs of the first rot dims turned, the rest as it was."""
    rot = case["rot"]
    y = x.clone()
    if case["style"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _quantize(x):
    """Q8_0 blocks of x [..., hd]: codes, rounded half away from zero, and scales."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127
    y = b * torch.where(d > 0, 1 / d, 0.0)
    code = torch.copysign(torch.floor(y.abs() + 0.5), y).clamp(-127, 127)
    return code.flatten(-2).to(torch.int8), d[..., 0].to(torch.float16)


def _store(s):
    case = s["case"]
    nh, nkv, hd, rows, P = case["nh"], case["nkv"], case["hd"], case["rows"], case["page"]
    x = s["qkv"].float()
    if s["bias"] is not None:
        x = x + s["bias"]
    x = x.view(rows, nh + 2 * nkv, hd)
    q, k, v = x[:, :nh], x[:, nh:nh + nkv], x[:, nh + nkv:]
    if s["q_norm"] is not None:
        norm = lambda y, w: y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
        q, k = norm(q, s["q_norm"]), norm(k, s["k_norm"])
    f, scale = _frequencies(case, x.device)
    angle = s["pos"].double()[:, None] * f
    cos, sin = ((g(angle) * scale).float()[:, None] for g in (torch.cos, torch.sin))
    live = (s["slot"] >= 0)[:, None]
    s["out"].copy_(torch.where(live, _turn(q, cos, sin, case).reshape(rows, -1).to(s["out"].dtype), s["out"]))
    # padding rows write what the first row does
    pick = torch.where(s["slot"] >= 0, torch.arange(rows, device=x.device), 0)
    slot = s["slot"].long()[pick]
    for rows_of, codes, scales in ((_turn(k, cos, sin, case), s["k"], s["ks"]), (v, s["v"], s["vs"])):
        c, d = _quantize(rows_of)
        codes[slot // P, slot % P] = c[pick]
        scales[slot // P, slot % P] = d[pick]
    back = lambda codes, scales: _values(codes, scales).to(torch.float16).reshape(-1, nkv * hd)  # noqa: E731
    return dict(q=s["out"], k=back(s["k"], s["ks"]), v=back(s["v"], s["vs"]))


def _read(s):
    case = s["case"]
    slot, P = s["slot"].long(), case["page"]
    one = lambda codes, scales: _values(codes[slot // P, slot % P], scales[slot // P, slot % P]).flatten(1).to(TYPES[case["type"]])  # noqa: E731
    return dict(k=one(s["k"], s["ks"]), v=one(s["v"], s["vs"]))


def _attention(s):
    case = s["case"]
    n, nh, nkv, hd, P = case["n"], case["nh"], case["nkv"], case["hd"], case["page"]
    j = torch.arange(case["max_len"], device="cuda")
    live = j[None, :] < s["length"][:, None]
    page = torch.where(live, s["table"][:, j // P], 0).long()
    row = (j % P)[None, :]
    k, v = (_values(s[c][page, row], s[d][page, row]) for c, d in (("k", "ks"), ("v", "vs")))  # [n, L, nkv, hd]
    q = s["q"].float().view(n, nkv, nh // nkv, hd)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1 / math.sqrt(hd))
    score.masked_fill_(~live[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    return dict(o=o.reshape(n, nh * hd).to(s["q"].dtype), lse=(torch.log(total) + top).view(n, nh))


def _sample(s):
    V = s["x"].shape[1]
    col = lambda x: x.double()[:, None]  # noqa: E731
    x = s["x"].double()
    best, order = torch.sort(x, dim=-1, descending=True, stable=True)
    top = best[:, :1]
    none = torch.isneginf(top)
    greedy = col(s["temperature"]) == 0
    temp = torch.where(greedy, 1.0, col(s["temperature"]))
    sharp = temp if s["case"]["first"] else 1.0  # the temperature that the filters see
    z = best - torch.where(none, 0.0, top)
    # the filters, in descending order
    rank = torch.arange(V, device=x.device)
    kept = rank < torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    w = torch.where(kept, torch.exp(z / sharp), 0.0)
    mass = w.cumsum(-1)
    p = col(s["top_p"])
    kept &= (p >= 1) | (mass - w < p * mass[:, -1:])
    kept &= z / sharp >= torch.log(col(s["min_p"]))
    kept &= (z / temp >= -60 * math.log(2)) & ~none
    kept = torch.where(greedy, rank == 0, kept | ((rank == 0) & ~none))
    # the draw, in the tokens' own order
    kept = torch.zeros_like(kept).scatter_(1, order, kept)
    w = torch.where(kept, torch.exp((x - torch.where(none, 0.0, top)) / temp), 0.0)
    mass = w.cumsum(-1)
    token = (mass <= col(s["u"]) * mass[:, -1:]).sum(-1, keepdim=True).clamp(max=V - 1)
    logprob = torch.log(w.gather(1, token)) - torch.log(mass[:, -1:])
    return dict(token=torch.where(none, -1, token)[:, 0].to(torch.int32), logprob=torch.where(none, -math.inf, logprob)[:, 0].float())


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import quantized_transformer_prefill_gb300 as qp
    op = s["case"]["op"]
    if op == "store":
        q = qp.op_rope_paged_store_q8(s["qkv"], s["rope"], s["pos"], s["slot"], s["cache"], s["case"]["nh"], bias=s["bias"],
                                      q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, out=s["out"])
        k, v = qp.op_paged_read_q8(s["cache"], s["every"], out=s["back"])
        return dict(q=q, k=k, v=v)
    if op == "read":
        k, v = qp.op_paged_read_q8(s["cache"], s["slot"], out=s["out"])
        return dict(k=k, v=v)
    if op == "attention":
        o = qp.op_paged_attention_q8(s["q"], s["cache"], s["table"], s["length"], s["case"]["nh"], out=s["out"], lse=s["lse"], workspace=s["work"])
        return dict(o=o, lse=s["lse"])
    token, logprob = qp.op_sample(s["x"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], temperature_first=s["case"]["first"],
                                  out=s["out"])
    return dict(token=token, logprob=logprob)


def run(s):
    if own:
        return _own(s)
    return {"store": _store, "read": _read, "attention": _attention, "sample": _sample}[s["case"]["op"]](s)


# ------------------------------------------------------------------ work
def work(case):
    """What a pass cannot do without.  Ragged lengths are uniform below max_len: their mean counts."""
    op = case["op"]
    if op == "sample":
        return dict(bytes=case["rows"] * (case["vocab"] * SIZE[case["type"]] + 28), flops=2 * case["rows"] * case["vocab"])
    nkv, hd, P = case["nkv"], case["hd"], case["page"]
    row = 2 * nkv * (hd + hd // 16)  # of K and V, codes and scales
    if op == "store":
        rows, nh = case["rows"] - case["pad"], case["nh"]
        pool = (-(-case["rows"] // P) + 3) * P
        return dict(bytes=rows * ((nh + 2 * nkv) * hd * SIZE[case["src"]] + nh * hd * SIZE[case["to"]] + row + 8) + (4 * (nh + 2 * nkv) * hd if case["bias"] else 0)
                    + pool * (row + 4 * nkv * hd + 4), flops=3 * rows * (nh + nkv) * case["rot"] + 4 * rows * 2 * nkv * hd)
    if op == "read":
        return dict(bytes=case["rows"] * (row + 2 * nkv * hd * SIZE[case["type"]] + 4), flops=case["rows"] * 2 * nkv * hd)
    n, nh = case["n"], case["nh"]
    keys = n * case["max_len"] * (1.0 if case["lens"] == "same" or n == 1 else 0.5)
    return dict(bytes=keys * row + 2 * n * nh * hd * SIZE[case["type"]] + 4 * n * nh + 4 * keys / P, flops=4 * keys * nh * hd)


# ------------------------------------------------------------------ the same from the definitions, in 64 bits
def _blocks(codes, scales):
    return codes.double() * scales.double().repeat_interleave(32, -1)


def _exact_store(s):
    case = s["case"]
    nh, nkv, hd, rot, P = case["nh"], case["nkv"], case["hd"], case["rot"], case["page"]
    f, scale = _frequencies(case, "cuda")
    live = s["slot"] >= 0
    x = s["qkv"].double()[live]
    if s["bias"] is not None:
        x = x + s["bias"].double()
    x = x.view(x.shape[0], nh + 2 * nkv, hd)
    if s["q_norm"] is not None:
        w = torch.cat([s["q_norm"].double().expand(nh, hd), s["k_norm"].double().expand(nkv, hd)])
        y = x[:, :nh + nkv]
        x = torch.cat([y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w, x[:, nh + nkv:]], 1)
    # a pair as a complex number, times e^(i angle)
    turn = torch.polar(torch.full_like(f, scale).expand(x.shape[0], -1), s["pos"][live].double()[:, None] * f)[:, None]
    y = x[:, :nh + nkv, :rot]
    if case["style"] == "half":
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:].contiguous()) * turn
        y = torch.cat([z.real, z.imag], -1)
    else:
        y = torch.view_as_real(torch.view_as_complex(y.reshape(y.shape[0], nh + nkv, rot // 2, 2).contiguous()) * turn).flatten(-2)
    y = torch.cat([y, x[:, :nh + nkv, rot:]], -1)
    q = s["out"].double()
    q[live] = y[:, :nh].reshape(-1, nh * hd)
    at = s["slot"][live].long()
    got = dict(q=q)
    for name, new in (("k", y[:, nh:]), ("v", x[:, nh + nkv:])):
        d = torch.linalg.vector_norm(new.reshape(*new.shape[:-1], hd // 32, 32), ord=math.inf, dim=-1).repeat_interleave(32, -1) / 127
        code = torch.where(d > 0, (new / d).abs().add(0.5).floor() * new.sign(), 0.0)
        pool = _blocks(s[name], s[name + "s"])
        pool[at // P, at % P] = code * d.half().double()
        got[name] = pool.reshape(-1, nkv * hd)
    return got


def _exact_read(s):
    P = s["case"]["page"]
    at = s["slot"].long()
    page = torch.div(at, P, rounding_mode="floor")
    return {name: torch.cat([_blocks(s[name][p, r], s[name + "s"][p, r]).flatten(1) for p, r in zip(page.split(8192), (at - page * P).split(8192))])
            for name in ("k", "v")}


def _exact_attention(s):
    case = s["case"]
    nh, nkv, hd, P = case["nh"], case["nkv"], case["hd"], case["page"]
    o = torch.zeros(case["n"], nh, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((case["n"], nh), -math.inf, dtype=torch.float64, device="cuda")
    for r, m in enumerate(s["length"].tolist()):
        if not m:
            continue
        pages = s["table"][r, :(m + P - 1) // P].long()
        k, v = (_blocks(s[c][pages], s[c + "s"][pages]).reshape(-1, nkv, hd)[:m] for c in ("k", "v"))
        q = s["q"][r].double().view(nkv, nh // nkv, hd)
        score = torch.einsum("hgd,jhd->hgj", q, k) / math.sqrt(hd)
        z = torch.logsumexp(score, -1)
        lse[r] = z.flatten()
        o[r] = torch.einsum("hgj,jhd->hgd", torch.exp(score - z[..., None]), v).reshape(nh, hd)
    return dict(o=o.view(case["n"], nh * hd), lse=lse)


def _exact_sample(s):
    """Request by request, on lists of the tokens that are left."""
    rows, V = s["x"].shape
    tokens, logprobs = [], []
    settings = zip(*(s[k].tolist() for k in ("temperature", "top_k", "top_p", "min_p", "u")))
    for r, (temp, k, p, floor, u) in enumerate(settings):
        x = s["x"][r].double()
        at = torch.nonzero(x > -math.inf)[:, 0]
        if not len(at):
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        if temp == 0:
            tokens.append(int(torch.nonzero(x == x.max())[0, 0]))
            logprobs.append(0.0)
            continue
        sharp = temp if s["case"]["first"] else 1.0
        at = at[torch.argsort(-x[at], stable=True)][:k if k > 0 else V]
        share = torch.softmax(x[at] / sharp, 0)
        n = len(at)
        if p < 1:
            n = max(1, int((share.cumsum(0) - share < p).sum()))
        share = share[:n]
        if floor > 0:
            n = max(1, int((share >= floor * share[0]).sum()))
        at = at[:n]
        at = at[(x[at] - x[at[0]]) / temp >= -60 * math.log(2)].sort().values
        logp = torch.log_softmax(x[at] / temp, 0)
        i = min(int((torch.cumsum(logp.exp(), 0) <= u * logp.exp().sum()).sum()), len(at) - 1)
        tokens.append(int(at[i]))
        logprobs.append(float(logp[i]))
    return dict(token=torch.tensor(tokens, dtype=torch.int32), logprob=torch.tensor(logprobs, dtype=torch.float64))


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](s)
