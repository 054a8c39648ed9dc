"""The operators of a served batch, as they are measured: cases, inputs, plain forms and 64-bit values.

One decode step of a batch of requests over a paged key-value cache runs them in this order:

  pages      block tables and slot maps from the requests' lengths
  rope       bias, QK-norm and rotary positions of the fused Q|K|V rows; K and V stored at their slots
  attention  one new token per request over its pages
  logprobs   log probability of given tokens, entropy and top alternatives of logits rows

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
        # one decode step of a small batch: every request gets one token (latency)
        dict(name="pages decode 32", op="pages", n=32, page=16, max_len=4096, mix="decode"),
        # a busy scheduler step: new prompts, rollbacks of rejected drafts, requests that end, and single tokens
        dict(name="pages mixed 1023", op="pages", n=1023, page=64, max_len=2048, mix="mixed"),
        # decode step of a batch, fused Q|K|V rows straight from a 16-bit projection
        dict(name="rope decode 64", op="rope", rows=64, nh=14, nkv=2, hd=64, src="bf16", to="bf16", page=16, style="half",
             rot=64, scaling="none", norm=False, bias=True, first=700, pad=0),
        # a long prompt chunk of the widest layout, f32 sums of the quantized GEMM into a bf16 cache, positions past the trained context
        dict(name="rope prefill 4096 yarn", op="rope", rows=4096, nh=28, nkv=4, hd=128, src="f32", to="bf16", page=16,
             style="half", rot=128, scaling="yarn", norm=False, bias=True, first=60000, pad=0),
        # a ragged chunk with QK-norm, half of each head rotated in interleaved pairs, padding rows at the end of a captured step
        dict(name="rope norm 1001", op="rope", rows=1001, nh=16, nkv=8, hd=128, src="f16", to="f16", page=32,
             style="interleaved", rot=64, scaling="linear", norm=True, bias=False, first=3, pad=23),
        # one request after a 512-token prompt (latency, split over the length)
        dict(name="attention 1 x 513", op="attention", n=1, lens="same", max_len=513, nh=14, nkv=2, hd=64, type="bf16", page=16, order="rows"),
        # a full serving batch, lengths spread up to 4096, one empty request
        dict(name="attention 64 x 4096", op="attention", n=64, lens="ragged", max_len=4096, nh=28, nkv=4, hd=128, type="bf16", page=16, order="rows"),
        # one very long context
        dict(name="attention 1 x 131071", op="attention", n=1, lens="same", max_len=131071, nh=12, nkv=2, hd=128, type="f16", page=64, order="heads"),
        # f32 pages, as the framework's own regions hold them
        dict(name="attention 33 x 2048 f32", op="attention", n=33, lens="ragged", max_len=2048, nh=14, nkv=2, hd=64, type="f32", page=32, order="rows"),
        # the token of one decode step with its alternatives (latency)
        dict(name="logprobs 1 x 151936", op="logprobs", rows=1, vocab=151936, type="f32", k=5, masked=False, extra=0),
        # every prompt row scored
        dict(name="logprobs 512 x 151936", op="logprobs", rows=512, vocab=151936, type="f32", k=20, masked=False, extra=0),
        # 16-bit logits of a batch under a grammar mask, odd vocabulary and row stride, one row with nothing left
        dict(name="logprobs 65 x 150001", op="logprobs", rows=65, vocab=150001, type="bf16", k=8, masked=True, extra=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "rope", "attention", "attention", "attention", "logprobs", "logprobs"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    nh, nkv, hd = rng.choice(HEADS)
    if op == "pages":
        n = _log(rng, 1, 2000)
        return dict(op=op, n=n, page=max(page, 8), max_len=_log(rng, 64, min(8192, max(64, 2000000 // n))), mix=rng.choice(["decode", "mixed", "mixed"]))
    if op == "rope":
        src, to = rng.choice([("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
        norm = rng.random() < 0.4
        rows = _log(rng, 1, 2048 if src == "f32" else 4096)
        return dict(op=op, rows=rows, nh=nh, nkv=nkv, hd=hd, src=src, to=to, page=page, style=rng.choice(["half", "interleaved"]),
                    rot=rng.choice([hd, hd, hd // 2, hd // 4, 24]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]), norm=norm,
                    bias=not norm, first=_log(rng, 1, 1000000), pad=rng.choice([0, 0, rng.randrange(0, rows)]))
    if op == "attention":
        t = rng.choice(["f32", "f16", "bf16", "bf16"])
        length = _log(rng, 1, 100000)
        most = max(1, min(256, 64 * 4096 * 4 * 128 * 2 // (length * nkv * hd * SIZE[t])))
        return dict(op=op, n=_log(rng, 1, most), lens=rng.choice(["same", "ragged", "ragged"]), max_len=length, nh=nh, nkv=nkv, hd=hd, type=t,
                    page=page, order=rng.choice(["rows", "heads"]))
    vocab = rng.choice([4096, 151936, 152064, _log(rng, 33, 152064)])
    t = rng.choice(["f32", "f32", "f16", "bf16"])
    return dict(op=op, rows=_log(rng, 1, min(4096, 512 * 151936 // vocab)), vocab=vocab, type=t, k=rng.choice([0, 1, 5, 20, 32]),
                masked=rng.random() < 0.4, extra=rng.choice([0, 0, 1, 7, 64]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lens(case, g):
    """Request lengths on the host: all of max_len, or spread below it with one empty request."""
    n, top = case["n"], case["max_len"]
    if case["lens"] == "same":
        return torch.full((n,), top, dtype=torch.int32)
    x = torch.randint(1, top + 1, (n,), generator=g, device="cuda", dtype=torch.int32).cpu()
    x[n // 2] = 0
    x[0] = top
    return x


def _prepare_pages(case, g):
    n, P, W = case["n"], case["page"], -(-case["max_len"] // case["page"])
    top = W * P
    length = torch.randint(0, top // 2 + 1, (n,), generator=g, device="cuda")
    target = length + 1
    if case["mix"] == "mixed":
        what = torch.randint(0, 16, (n,), generator=g, device="cuda")
        some = torch.randint(1, max(2, top // 8), (n,), generator=g, device="cuda")
        length = torch.where(what < 1, 0, length)
        target = torch.where(what < 2, length + some, torch.where(what == 2, (length - some % 8).clamp(min=0), torch.where(what == 3, 0, length + 1)))
    # a step of a fixed size, as a captured graph has it: a budget of new tokens, the rows behind the last one are padding
    most = n + 1 + n // 16 if case["mix"] == "decode" else 64 + n * (1 + top // 100)
    count = (target - length).clamp(min=0)
    target = torch.where(count > 0, length + torch.minimum(count, (most - count.cumsum(0) + count).clamp(min=0)), target)
    held, n_pages = -(-length // P), n * W
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, W), -1, dtype=torch.int32, device="cuda")
    mine = torch.arange(W, device="cuda")[None, :] < held[:, None]
    total = int(held.sum())
    table[mine] = ids[:total]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_pages - total] = ids[total:]
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(length=length.to(torch.int32), target=target.to(torch.int32), table=table, free=free, n_pages=n_pages, max_tokens=most,
                n_free=torch.tensor([n_pages - total], dtype=torch.int32, device="cuda"), out=(i32(n + 1), i32(most), i32(most), i32(1)))


def _rope_args(case):
    kind = case["scaling"]
    return dict(rot_dim=case["rot"], theta=1.0e6, style=case["style"], scaling=kind, factor=1.0 if kind == "none" else 4.0,
                n_ctx_orig=32768 if kind == "yarn" else 0)


def _prepare_rope(case, g):
    rows, nh, nkv, hd, P = case["rows"], case["nh"], case["nkv"], case["hd"], case["page"]
    width = (nh + 2 * nkv) * hd
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n_pages = -(-rows // P) + 3
    pool = lambda: new(n_pages, P, nkv, hd).to(TYPES[case["to"]])  # noqa: E731
    pos = torch.arange(rows, device="cuda", dtype=torch.int32) + case["first"]
    slot = torch.randperm(n_pages * P, generator=g, device="cuda")[:rows].to(torch.int32)
    live = rows - case["pad"]
    pos[live:] = -1
    slot[live:] = -1
    s = dict(qkv=(1.5 * new(rows, width)).to(TYPES[case["src"]]), pos=pos, slot=slot, k=pool(), v=pool(), bias=None, q_norm=None, k_norm=None,
             out=torch.zeros(rows, nh * hd, dtype=TYPES[case["to"]], device="cuda"))
    if case["bias"]:
        s["bias"] = 0.5 * new(width)
    if case["norm"]:
        s["q_norm"], s["k_norm"] = 1 + 0.1 * new(hd), 1 + 0.1 * new(hd)
    if own:
        import quantized_transformer_prefill_gb300 as qp
        s["cache"] = qp.PagedCache(s["k"], s["v"])
        s["rope"] = qp.RopeTable(hd, **_rope_args(case))
    return s


def _prepare_attention(case, g):
    n, nh, nkv, hd, P = case["n"], case["nh"], case["nkv"], case["hd"], case["page"]
    t, W = TYPES[case["type"]], -(-case["max_len"] // P)
    length = _lens(case, g).cuda()
    held = -(-length.long() // P)
    n_pages = int(held.sum()) + 2
    table = torch.full((n, W), -1, dtype=torch.int32, device="cuda")
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table[torch.arange(W, device="cuda")[None, :] < held[:, None]] = ids[:n_pages - 2]
    # rows of all heads behind one another, or each head's rows of a page behind one another
    shape = (n_pages, P, nkv, hd) if case["order"] == "rows" else (n_pages, nkv, P, hd)
    pool = lambda: torch.randn(*shape, generator=g, device="cuda", dtype=t).permute(*((0, 1, 2, 3) if case["order"] == "rows" else (0, 2, 1, 3)))  # noqa: E731
    s = dict(q=(1.3 * torch.randn(n, nh * hd, generator=g, device="cuda")).to(t), k=pool(), v=pool(), table=table, length=length, nh=nh,
             out=torch.empty(n, nh * hd, dtype=t, device="cuda"), lse=torch.empty(n, nh, device="cuda"))
    if own:
        import quantized_transformer_prefill_gb300 as qp
        s["cache"] = qp.PagedCache(s["k"], s["v"])
        s["work"] = qp.op_paged_attention_workspace(s["cache"], n, nh)
    return s


def _prepare_logprobs(case, g):
    rows, V, t = case["rows"], case["vocab"], TYPES[case["type"]]
    x = torch.empty(rows, V + case["extra"], device="cuda", dtype=t)
    x.normal_(0.0, 2.5, generator=g)
    # a few likely tokens above the rest, as a trained model's head gives them
    likely = (torch.randint(0, V, (rows, 1), generator=g, device="cuda") + torch.arange(6, device="cuda") * (V // 7)) % V
    x.scatter_(1, likely, (13 + 2 * torch.randn(rows, 6, generator=g, device="cuda")).to(t))
    ids = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.7, likely[:, 0], torch.randint(0, V, (rows,), generator=g, device="cuda"))
    if case["masked"]:
        x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < 0.5, -math.inf)
        x[rows // 2].fill_(-math.inf)
    k = case["k"]
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    s = dict(x=x[:, :V], ids=ids.to(torch.int32), k=k, out=(f(rows), f(rows), torch.empty(rows, k, dtype=torch.int32, device="cuda"), f(rows, k)))
    if own:
        import quantized_transformer_prefill_gb300 as qp
        s["work"] = qp.op_token_logprobs_workspace(s["x"], k)
    return s


def prepare(case, seed):
    s = {"pages": _prepare_pages, "rope": _prepare_rope, "attention": _prepare_attention, "logprobs": _prepare_logprobs}[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _pages(s):
    P, W = s["case"]["page"], s["table"].shape[1]
    length, target, table, free, n_free = s["length"].long(), s["target"].long(), s["table"], s["free"], s["n_free"]
    held, need = (length + P - 1) // P, (target + P - 1) // P
    col = torch.arange(W, device=table.device)[None, :]
    gone = (col >= need[:, None]) & (col < held[:, None])
    come = (col >= held[:, None]) & (col < need[:, None])
    # the stack of free pages with the returned ones on top: entry i lies in the list below n_free, in `back` above
    back = torch.full((table.numel() + 1,), -1, dtype=torch.int32, device=table.device)
    at = torch.where(gone, gone.flatten().cumsum(0).view_as(gone) - 1, table.numel())
    back.scatter_(0, at.flatten(), table.flatten())
    size = n_free.long() + gone.sum()
    nth = come.flatten().cumsum(0).view_as(come) - 1
    i = size - 1 - nth
    took = torch.where(i < n_free, free[i.clamp(0, free.numel() - 1)], back[(i - n_free).clamp(0, table.numel())])
    table.copy_(torch.where(come, took, table))
    left = size - come.sum()
    j = torch.arange(free.numel(), device=table.device)
    free.copy_(torch.where((j >= n_free) & (j < left), back[(j - n_free).clamp(0, table.numel())], free))
    count = (target - length).clamp(min=0)
    start = torch.cat([count.new_zeros(1), count.cumsum(0)])
    t = torch.arange(s["max_tokens"], device=table.device)
    r = torch.searchsorted(start, t, right=True) - 1
    live = t < start[-1]
    r = torch.where(live, r, 0)
    pos = t - start[r] + length[r]
    slot = table[r, (pos // P).clamp(0, W - 1)].long() * P + pos % P
    i32 = torch.int32
    return dict(table=table, free=free, n_free=left.to(i32).view(1), start=start.to(i32), pos=torch.where(live, pos, -1).to(i32),
                slot=torch.where(live, slot, -1).to(i32))


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


def _rope(s):
    case = s["case"]
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    rows = case["rows"]
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
    t = s["k"].dtype
    live = (s["slot"] >= 0)[:, None]
    s["out"].copy_(torch.where(live, _turn(q, cos, sin, case).reshape(rows, -1).to(t), s["out"]))
    # padding rows write what the first row does
    pick = torch.where(s["slot"] >= 0, torch.arange(rows, device=x.device), 0)
    slot = s["slot"].long()[pick]
    P = case["page"]
    s["k"][slot // P, slot % P] = _turn(k, cos, sin, case).to(t)[pick]
    s["v"][slot // P, slot % P] = v.to(t)[pick]
    return dict(q=s["out"], k=s["k"], v=s["v"])


def _attention(s):
    case = s["case"]
    n, nh, nkv, hd, P = case["n"], case["nh"], case["nkv"], case["hd"], case["page"]
    L = case["max_len"]
    j = torch.arange(L, device="cuda")
    live = j[None, :] < s["length"][:, None]
    page = torch.where(live, s["table"][:, j // P], 0).long()
    k, v = (x[page, (j % P)[None, :]].float() for x in (s["k"], s["v"]))  # [n, L, nkv, hd]
    q = s["q"].float().view(n, nkv, nh // nkv, hd)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1 / math.sqrt(hd))
    score.masked_fill_(~live[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    return dict(o=o.reshape(n, nh * hd).to(s["q"].dtype), lse=(torch.log(total) + top).view(n, nh))


def _logprobs(s):
    x, k = s["x"].float(), s["k"]
    top = x.amax(-1, keepdim=True)
    none = top == -math.inf
    base = torch.where(none, 0.0, top)
    e = torch.exp(x - base)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total) + base
    mean = torch.where(e > 0, e * (x - base), 0.0).sum(-1, keepdim=True) / total
    entropy = torch.where(none, 0.0, torch.log(total) - mean)[:, 0]
    order = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :k]
    of = lambda i: torch.where(none, -math.inf, x.gather(1, i.long()) - lse)  # noqa: E731
    return dict(logprob=of(s["ids"][:, None])[:, 0], entropy=entropy, top_ids=order.to(torch.int32), top_logprobs=of(order))


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import quantized_transformer_prefill_gb300 as qp
    op = s["case"]["op"]
    if op == "pages":
        start, pos, slot, n_free = qp.op_page_tables(s["length"], s["target"], s["case"]["page"], s["table"], s["free"], s["n_free"],
                                                     s["n_pages"], s["max_tokens"], out=s["out"])
        return dict(table=s["table"], free=s["free"], n_free=n_free, start=start, pos=pos, slot=slot)
    if op == "rope":
        q = qp.op_rope_paged_store(s["qkv"], s["rope"], s["pos"], s["slot"], s["cache"], s["case"]["nh"], bias=s["bias"],
                                   q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, out=s["out"])
        return dict(q=q, k=s["k"], v=s["v"])
    if op == "attention":
        o = qp.op_paged_attention(s["q"], s["cache"], s["table"], s["length"], s["nh"], out=s["out"], lse=s["lse"], workspace=s["work"])
        return dict(o=o, lse=s["lse"])
    logprob, entropy, top_ids, top_logprobs = qp.op_token_logprobs(s["x"], s["ids"], s["k"], out=s["out"], workspace=s["work"])
    return dict(logprob=logprob, entropy=entropy, top_ids=top_ids, top_logprobs=top_logprobs)


def run(s):
    if own:
        return _own(s)
    return {"pages": _pages, "rope": _rope, "attention": _attention, "logprobs": _logprobs}[s["case"]["op"]](s)


# ------------------------------------------------------------------ work
def work(case):
    """What a pass cannot do without.  Ragged lengths are uniform below max_len: their mean counts."""
    op = case["op"]
    if op == "pages":
        n, P = case["n"], case["page"]
        top = -(-case["max_len"] // P) * P
        # mixed: 2/16 of the requests add top/16 tokens on average, 12/16 one; decode: one each
        tokens = n if case["mix"] == "decode" else n * (2 / 16 * max(1, top // 16) + 12 / 16)
        return dict(bytes=4 * (2 * n + (n + 1) + 2 * tokens + 2 * n + 2 * tokens / P), flops=0)
    if op == "rope":
        rows, width = case["rows"] - case["pad"], (case["nh"] + 2 * case["nkv"]) * case["hd"]
        turned = rows * (case["nh"] + case["nkv"]) * case["rot"]
        return dict(bytes=rows * (width * (SIZE[case["src"]] + SIZE[case["to"]]) + 8) + (4 * width if case["bias"] else 0), flops=3 * turned)
    if op == "attention":
        n, nh, nkv, hd = case["n"], case["nh"], case["nkv"], case["hd"]
        keys = n * case["max_len"] * (1.0 if case["lens"] == "same" or n == 1 else 0.5)
        return dict(bytes=keys * 2 * nkv * hd * SIZE[case["type"]] + 2 * n * nh * hd * SIZE[case["type"]] + 4 * n * nh + 4 * keys / case["page"],
                    flops=4 * keys * nh * hd)
    return dict(bytes=case["rows"] * (case["vocab"] * SIZE[case["type"]] + 12 + 8 * case["k"]), flops=4 * case["rows"] * case["vocab"])


# ------------------------------------------------------------------ the same from the definitions, in 64 bits
def _exact_pages(s):
    P = s["case"]["page"]
    length, target, table, free = s["length"].tolist(), s["target"].tolist(), s["table"].tolist(), s["free"].tolist()
    stack = free[:int(s["n_free"])]
    pages = lambda m: (m + P - 1) // P  # noqa: E731
    for r, (a, b) in enumerate(zip(length, target)):
        stack += table[r][pages(b):pages(a)]
    start, pos, slot = [0], [], []
    for r, (a, b) in enumerate(zip(length, target)):
        for i in range(pages(a), pages(b)):
            table[r][i] = stack.pop()
        pos += range(a, b)
        slot += [table[r][p // P] * P + p % P for p in range(a, b)]
        start.append(len(pos))
    free[int(s["n_free"]):len(stack)] = stack[int(s["n_free"]):]
    rest = [-1] * (s["max_tokens"] - len(pos))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return dict(table=i32(table), free=i32(free), n_free=i32([len(stack)]), start=i32(start), pos=i32(pos + rest), slot=i32(slot + rest))


def _exact_rope(s):
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
    q, k, v = s["out"].double(), s["k"].double(), s["v"].double()
    q[live] = y[:, :nh].reshape(-1, nh * hd)
    at = s["slot"][live].long()
    k[at // P, at % P] = y[:, nh:]
    v[at // P, at % P] = x[:, nh + nkv:]
    return dict(q=q, k=k, v=v)


def _exact_attention(s):
    case = s["case"]
    nh, nkv, hd, P = case["nh"], case["nkv"], case["hd"], case["page"]
    o = torch.zeros(case["n"], nh, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((case["n"], nh), -math.inf, dtype=torch.float64, device="cuda")
    for r, m in enumerate(s["length"].tolist()):
        if not m:
            continue
        pages = s["table"][r, :(m + P - 1) // P].long()
        k, v = (x[pages].reshape(-1, nkv, hd)[:m].double() for x in (s["k"], s["v"]))
        q = s["q"][r].double().view(nkv, nh // nkv, hd)
        score = torch.einsum("hgd,jhd->hgj", q, k) / math.sqrt(hd)
        z = torch.logsumexp(score, -1)
        lse[r] = z.flatten()
        o[r] = torch.einsum("hgj,jhd->hgd", torch.exp(score - z[..., None]), v).reshape(nh, hd)
    return dict(o=o.view(case["n"], nh * hd), lse=lse)


def _exact_logprobs(s):
    got = []
    for x, i in zip(s["x"].split(64), s["ids"].split(64)):
        x = x.double()
        lse = torch.logsumexp(x, -1, keepdim=True)
        dead = torch.isneginf(lse)
        logp = torch.where(dead, -math.inf, x - lse)
        entropy = torch.special.entr(torch.where(dead, 0.0, logp.exp())).sum(-1)
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :s["k"]]
        got.append((logp.gather(1, i.long()[:, None])[:, 0], entropy, order.to(torch.int32), logp.gather(1, order)))
    return dict(zip(("logprob", "entropy", "top_ids", "top_logprobs"), (torch.cat(x) for x in zip(*got))))


def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "rope": _exact_rope, "attention": _exact_attention, "logprobs": _exact_logprobs}[case["op"]](s)
