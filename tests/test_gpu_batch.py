"""The batch operators on the GPU against plain 64-bit implementations: page
tables and slot maps, RoPE with the paged store, paged attention of one token
per request, token log probabilities, and a run of them together.

Whole numbers are equal.  Float tolerances count roundings: U is the f32 unit
roundoff, half(t) = finfo(t).eps / 2 the one of a stored type."""
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32


def half(t):
    return torch.finfo(t).eps / 2


@pytest.fixture(scope="module")
def qp():
    import quantized_transformer_prefill_gb300 as qp
    qp.lib()
    return qp


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def status_word():
    return torch.zeros(1, dtype=I32, device="cuda")


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def close(got, want, tol):
    """|got - want| <= tol elementwise, equal where want is not finite."""
    got, want = got.double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine].nan_to_num(nan=7e7), want[~fine].nan_to_num(nan=7e7))
    tol = torch.as_tensor(tol, dtype=torch.float64, device=got.device).expand_as(want)
    off = (got - want).abs()
    bad = fine & ~(off <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / tol)[bad].max()):.3g} of the tolerance"


# ------------------------------------------------------------------ page tables
def tables_by_hand(length, target, P, table, free, n_free, max_tokens):
    """The definition, on lists; None where the step is refused."""
    table, free = [list(r) for r in table], list(free)
    stack = free[:n_free]
    n = lambda m: -(-m // P)  # noqa: E731
    for r, (a, b) in enumerate(zip(length, target)):
        stack += table[r][n(b):n(a)] if b < a else []
    start, pos, slot = [0], [], []
    for r, (a, b) in enumerate(zip(length, target)):
        for i in range(n(a), n(b)):
            if not stack:
                return None
            table[r][i] = stack.pop()
        for p in range(a, b):
            pos.append(p)
            slot.append(table[r][p // P] * P + p % P)
        start.append(len(pos))
    if len(pos) > max_tokens:
        return None
    free[n_free:len(stack)] = stack[n_free:]
    rest = [-1] * (max_tokens - len(pos))
    return table, free, len(stack), start, pos + rest, slot + rest


def tables_case(seed, n, P, W, kinds):
    rng = random.Random(seed)
    ids = list(range(n * W))
    rng.shuffle(ids)
    length, target, table = [], [], []
    for r in range(n):
        kind = rng.choice(kinds)
        a = 0 if kind == "new" else rng.randint(0, W * P)
        b = {"new": rng.randint(0, W * P), "one": min(a + 1, W * P), "over": 0, "back": max(0, a - rng.randint(0, P + 2)),
             "same": a, "grow": rng.randint(a, W * P)}[kind]
        held = -(-a // P)
        table.append([ids.pop() for _ in range(held)] + [-7] * (W - held))
        length.append(a)
        target.append(b)
    free = ids + [-1] * (n * W - len(ids))
    return length, target, table, free, len(ids)


def run_tables(qp, case, P, max_tokens, in_place=False, status=None):
    length, target, table, free, n_free = case
    t, f, nf = dev(table), dev(free), dev([n_free])
    out = (torch.full((len(length) + 1,), -9, dtype=I32, device="cuda"), torch.full((max_tokens,), -9, dtype=I32, device="cuda"),
           torch.full((max_tokens,), -9, dtype=I32, device="cuda"), nf if in_place else dev([-9]))
    start, pos, slot, left = qp.op_page_tables(dev(length), dev(target), P, t, f, nf, len(free), max_tokens, out=out, status=status)
    return t.tolist(), f.tolist(), int(left), start.tolist(), pos.tolist(), slot.tolist()


@pytest.mark.parametrize("n,P,W", [(1, 16, 4), (3, 1, 5), (33, 24, 7), (1023, 16, 3), (1025, 8, 2), (5000, 3, 2), (16384, 2, 1)])
@pytest.mark.parametrize("kinds", [["one"], ["new", "one", "over", "back", "same", "grow"], ["over", "back"], ["same"]])
def test_page_tables(qp, n, P, W, kinds):
    case = tables_case(n * 7 + P, n, P, W, kinds)
    tokens = sum(max(0, b - a) for a, b in zip(*case[:2]))
    for max_tokens, in_place in ((tokens, True), (tokens + 37, False), (tokens + 5000, True)):
        status = status_word()
        got = run_tables(qp, case, P, max_tokens, in_place, status)
        assert got == tables_by_hand(*case[:2], P, *case[2:], max_tokens)
        assert int(status) == 0


@pytest.mark.parametrize("n", [3412, 3413, 4061, 4062, 4095, 4096])
def test_page_tables_around_the_default_shared_memory(qp, n):
    """Three counts of 4 bytes a request pass 40 KB at 3,413 requests and 48 KB, less the kernel's static bytes, from
    about 4,062: on either side of both the step is done."""
    test_page_tables(qp, n, 8, 2, ["one", "same", "back"])


def test_page_tables_long_prompt_into_an_empty_pool(qp):
    P, W = 128, 1024
    ids = list(range(2 * W))
    case = ([0, 5], [P * W, 6], [[-1] * W, [ids.pop()] + [-1] * (W - 1)], ids + [-1], len(ids))
    assert run_tables(qp, case, P, P * W + 1) == tables_by_hand(*case[:2], P, *case[2:], P * W + 1)


@pytest.mark.parametrize("n", [9, 3000])
@pytest.mark.parametrize("what,code", [("negative length", -2), ("negative target", -2), ("long length", -2), ("long target", -2), ("tokens", -10),
                                       ("pages", -7), ("depth", -1), ("negative depth", -1), ("free id", -1), ("shared page id", -1),
                                       ("returned id", -1), ("too many returned", -1)])
def test_page_tables_refusals_change_nothing(qp, n, what, code):
    P, W = 16, 3
    length, target, table, free, n_free = tables_case(4, n, P, W, ["one", "over", "back"])
    r = n // 2
    length[r], target[r] = 18, 19  # two pages held, the second one shared by the new row
    table[r] = [0, 1, -7]
    r2 = r + 1
    length[r2], target[r2] = 16, 17  # takes a new page, the first one popped below
    max_tokens = sum(max(0, b - a) for a, b in zip(length, target)) + 3
    if what == "negative length":
        length[r] = -1
    elif what == "negative target":
        target[r] = -5
    elif what == "long length":
        length[r] = P * W + 1
    elif what == "long target":
        target[r] = P * W + 1
    elif what == "tokens":
        max_tokens = 1
    elif what == "pages":
        length, target = [16] * n, [17] * n
        table = [[i, -7, -7] for i in range(n)]
        n_free = n - 1
        max_tokens = n
    elif what == "depth":
        n_free = len(free) + 1
    elif what == "negative depth":
        n_free = -1
    elif what == "free id":
        length, target = [16] * n, [17] * n
        table = [[i, -7, -7] for i in range(n)]
        free, n_free = [n + i for i in range(n - 1)] + [n * W] + [-1] * (2 * n), n
        max_tokens = n
    elif what == "shared page id":
        table[r][1] = n * W
    elif what == "returned id":
        length[r2], target[r2] = 30, 3
        table[r2] = [4, -1, -7]
    elif what == "too many returned":
        length, target, table = [P * W] * n, [0] * n, [[0] * W] * n
        n_free = 1
        max_tokens = 4
    status = status_word()
    t, f, left, start, pos, slot = run_tables(qp, (length, target, table, free, n_free), P, max_tokens, False, status)
    assert int(status) == code
    assert t == table and f == free and left == -9
    assert start == [0] * (n + 1) and pos == [-1] * max_tokens and slot == [-1] * max_tokens
    with pytest.raises(qp.MinferError):
        qp.check_status(status)


# ------------------------------------------------------------------ RoPE + paged store
def rope_frequencies(rot, theta, scaling, factor, ctx):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    scale = 1.0
    if scaling == "ntk" and rot > 2:
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        d = [rot * math.log(ctx / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (32, 1)]
        low, high = max(math.floor(d[0]), 0), min(math.ceil(d[1]), rot - 1)
        g = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / factor * g + f * (1 - g)
        scale = 0.1 * math.log(factor) + 1
    return f, scale


def rope_by_formula(qkv, nh, nkv, hd, pos, f, scale, style, bias=None, norms=None, eps=1e-6):
    """Q [n][nh][hd], K, V in 64 bits, and what bounds their f32 error."""
    n, rot = qkv.shape[0], 2 * f.shape[0]
    x = qkv.double()
    size = x.abs()
    if bias is not None:
        x = x + bias.double()
        size = size + bias.double().abs()
    x, size = x.view(n, nh + 2 * nkv, hd), size.view(n, nh + 2 * nkv, hd)
    if norms is not None:
        y = x[:, :nh + nkv]
        w = torch.cat([norms[0].double().expand(nh, hd), norms[1].double().expand(nkv, hd)])
        r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        x = torch.cat([y * r * w, x[:, nh + nkv:]], 1)
        size = torch.cat([size[:, :nh + nkv] * r * w.abs(), size[:, nh + nkv:]], 1)
    i = torch.arange(rot // 2, device="cuda")
    a, b = (i, i + rot // 2) if style == "half" else (2 * i, 2 * i + 1)
    ang = pos.double()[:, None, None] * f
    c, s = torch.cos(ang) * scale, torch.sin(ang) * scale
    y = x.clone()
    q = nh + nkv
    y[:, :q, a] = x[:, :q, a] * c - x[:, :q, b] * s
    y[:, :q, b] = x[:, :q, b] * c + x[:, :q, a] * s
    bound = size.clone()
    both = (size[:, :q, a] + size[:, :q, b]) * scale
    bound[:, :q, a] = both
    bound[:, :q, b] = both
    return y, bound


# Roundings of the f32 arithmetic per element, in units of U: the bias add 1, the norm's sum of hd squares (hd/32 + 5 adds and
# the squares: at most 10, halved by the root), rsqrt 2 ulp = 4, two products 2; cos and sin 2 ulp = 4 with their angle's
# rounding 2 and the scale 1; two products and an add 3.
ROPE_F32 = (1 + 10 + 4 + 2 + 4 + 2 + 1 + 3) * U


ROPE_CASES = [
    # nh, nkv, hd, src, to, page, style, rot, scaling, norm, bias
    (14, 2, 64, BF16, BF16, 16, "half", 64, "none", False, True),
    (14, 2, 64, F32, F32, 16, "interleaved", 64, "none", False, True),
    (12, 2, 128, F32, BF16, 1, "half", 128, "yarn", False, True),
    (16, 8, 128, F16, F16, 24, "interleaved", 64, "linear", True, False),
    (16, 8, 128, F32, F32, 32, "half", 24, "ntk", True, False),
    (4, 2, 64, F32, F16, 128, "half", 6, "none", True, True),
    (4, 4, 64, F32, F32, 7, "half", 2, "none", False, False),
    (5, 1, 128, BF16, BF16, 16, "half", 90, "linear", True, True),
    (40, 8, 128, F32, BF16, 16, "half", 128, "none", False, False),
    (160, 32, 128, F32, F16, 16, "interleaved", 90, "yarn", False, True),
    (3, 3, 64, F16, F16, 16, "half", 20, "none", True, True),
]


@pytest.mark.parametrize("nh,nkv,hd,src,to,P,style,rot,scaling,norm,bias", ROPE_CASES)
@pytest.mark.parametrize("n,order", [(1, "rows"), (37, "rows"), (130, "heads")])
def test_rope_paged_store(qp, nh, nkv, hd, src, to, P, style, rot, scaling, norm, bias, n, order):
    g = gen(n + hd)
    width = (nh + 2 * nkv) * hd
    # rows of a wider buffer, the result too
    qkv = torch.randn(n, width + 64, generator=g, device="cuda").to(src)[:, :width]
    b = torch.randn(width, generator=g, device="cuda") if bias else None
    norms = tuple(1 + 0.2 * torch.randn(hd, generator=g, device="cuda") for _ in range(2)) if norm else None
    pages = -(-n // P) + 2
    shape = (pages, P, nkv, hd) if order == "rows" else (pages, nkv, P, hd)
    view = lambda x: x if order == "rows" else x.permute(0, 2, 1, 3)  # noqa: E731
    k0, v0 = (view(torch.randn(*shape, generator=g, device="cuda").to(to)) for _ in range(2))
    k, v = view(torch.empty(shape, dtype=to, device="cuda")), view(torch.empty(shape, dtype=to, device="cuda"))
    k.copy_(k0), v.copy_(v0)
    pos = torch.randint(0, 2 ** 31 - 1, (n,), generator=g, device="cuda").to(I32)
    pos[0] = 0
    if n > 3:
        pos[1], pos[2], pos[3] = 1, 2 ** 31 - 1, 131071
    slot = torch.randperm(pages * P, generator=g, device="cuda")[:n].to(I32)
    pad = torch.zeros(n, dtype=torch.bool, device="cuda")
    pad[n // 3::5] = n > 1
    pos[pad], slot[pad] = -1, -1
    qkv[pad] = math.nan  # what a padding row holds is not looked at
    out = torch.full((n, nh * hd + 8), 7.0, dtype=to, device="cuda")[:, :nh * hd]
    ctx, factor, theta = 4096, 4.0, 1e6
    rope = qp.RopeTable(hd, rot, theta, style, scaling, 1.0 if scaling == "none" else factor, ctx)
    status = status_word()
    qp.op_rope_paged_store(qkv, rope, pos, slot, qp.PagedCache(k, v), nh, bias=b, q_norm=norms and norms[0], k_norm=norms and norms[1],
                           eps=1e-6, out=out, status=status)
    assert int(status) == 0
    f, scale = rope_frequencies(rot, theta, scaling, 1.0 if scaling == "none" else factor, ctx)
    live = ~pad
    want, bound = rope_by_formula(qkv[live], nh, nkv, hd, pos[live], f, scale, style, b, norms)
    # f is rounded to 53 bits, the angle of position 2^31 with it: 2^31 * 2^-52 radians
    tol = half(to) * want.abs() + (ROPE_F32 + 2.0 ** -21) * bound + torch.finfo(to).smallest_normal * half(to) * 2
    close(out[live].view(-1, nh, hd), want[:, :nh], tol[:, :nh])
    at = slot[live].long()
    close(k[at // P, at % P], want[:, nh:nh + nkv], tol[:, nh:nh + nkv])
    close(v[at // P, at % P], want[:, nh + nkv:], tol[:, nh + nkv:])
    # nothing else is touched
    assert (out[pad] == 7).all()
    k[at // P, at % P] = k0[at // P, at % P]
    v[at // P, at % P] = v0[at // P, at % P]
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_rope_passes_unrotated_values_through(qp):
    """V and the dims behind rot_dim are copied, infinities and all."""
    n, nh, nkv, hd = 3, 2, 1, 64
    g = gen(3)
    qkv = torch.randn(n, 4 * hd, generator=g, device="cuda")
    qkv[1, 40], qkv[2, 3 * hd + 5] = math.inf, -math.inf
    k, v = (torch.zeros(2, 4, nkv, hd, device="cuda") for _ in range(2))
    q = qp.op_rope_paged_store(qkv, qp.RopeTable(hd, 16), dev([5, 6, 7]), dev([0, 5, 2]), qp.PagedCache(k, v), nh)
    at = torch.tensor([0, 5, 2], device="cuda")
    assert torch.equal(v[at // 4, at % 4].view(n, hd), qkv[:, 3 * hd:])
    assert torch.equal(k[at // 4, at % 4].view(n, hd)[:, 16:], qkv[:, 2 * hd + 16:3 * hd])
    assert torch.equal(q.view(n, nh, hd)[..., 16:], qkv.view(n, 4, hd)[:, :nh, 16:])


def test_rope_refuses_rows_on_the_device(qp):
    """A slot past the pool or a negative position: that row is not written."""
    n, nh, nkv, hd, P = 4, 4, 2, 64, 4
    qkv = torch.randn(n, 8 * hd, device="cuda")
    k, v = (torch.full((2, P, nkv, hd), 3.0, device="cuda") for _ in range(2))
    out = torch.full((n, nh * hd), 3.0, device="cuda")
    for pos, slot in (([0, 1, 2, 3], [0, 8, 2, 3]), ([0, -1, 2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 2 ** 31 - 1, 2, 3])):
        k.fill_(3.0), v.fill_(3.0), out.fill_(3.0)
        status = status_word()
        qp.op_rope_paged_store(qkv, qp.RopeTable(hd), dev(pos), dev(slot), qp.PagedCache(k, v), nh, out=out, status=status)
        assert int(status) == -2
        assert (out[1] == 3).all() and not (out[[0, 2, 3]] == 3).any()
        kept = torch.tensor([r for r in range(2 * P) if r not in (0, 2, 3)], device="cuda")
        assert (k.view(-1, nkv * hd)[kept] == 3).all() and (v.view(-1, nkv * hd)[kept] == 3).all()
        assert torch.equal(v.view(-1, nkv * hd)[[0, 2, 3]], qkv[[0, 2, 3], 6 * hd:])


# ------------------------------------------------------------------ paged attention
def attention_by_definition(q, k, v, table, length, nh, scale):
    """o, lse in 64 bits with their a-priori error terms: (o, lse, mean of |v| under the softmax, score error, max |v|)."""
    n, nkv, hd, P = q.shape[0], k.shape[2], k.shape[3], k.shape[1]
    G = nh // nkv
    o = torch.zeros(n, nh, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((n, nh), -math.inf, dtype=torch.float64, device="cuda")
    mean, top, err = torch.zeros_like(o), torch.zeros_like(o), torch.zeros(n, nh, 1, dtype=torch.float64, device="cuda")
    for r, m in enumerate(length):
        if m <= 0:
            continue
        pages = table[r, :-(-m // P)].long()
        kk, vv = (x[pages].double().reshape(-1, nkv, hd)[:m] for x in (k, v))
        qq = q[r].double().view(nkv, G, hd)
        s = torch.einsum("hgd,jhd->hgj", qq, kk) * scale
        z = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - z)
        lse[r] = z.flatten()
        o[r] = torch.einsum("hgj,jhd->hgd", p, vv).reshape(nh, hd)
        mean[r] = torch.einsum("hgj,jhd->hgd", p, vv.abs()).reshape(nh, hd)
        top[r] = vv.abs().amax(0).repeat_interleave(G, 0)
        err[r] = (torch.einsum("hgd,jhd->hgj", qq.abs(), kk.abs()).amax(-1, keepdim=True) * scale).reshape(nh, 1)
    return o, lse, mean, err, top


def attention_tolerance(t, hd, length, want):
    """Score error: the MMA sums over the head's dims truncate (2^-23 of the
    partial sum each, hd / 8 + 2 of them); of f32 operands as hi + lo, |lo| <= 2^-11
    of the value, the product of the two lo (2^-22) and the bits that the MMA cuts
    from each lo (2^-10 of it, 2^-21) are left out: 2^-22 + 2 * 2^-21 = 20 U of a
    product; the scaled score's rounding and the exponential's 2 ulp come on top.
    Each weight's relative error is the score error twice (its own and the sum's);
    16-bit weights are rounded (half a step, or half of the smallest subnormal under
    a sum that is at least 1), f32 weights and values lose 20 U again; sums of up to
    64 + units adds."""
    o, lse, mean, size, top = want
    steps = hd // 8 + 2
    split = 20 * U if t == F32 else 0
    score = size * (steps * 2.0 ** -23 + split + 4 * U) + 8 * U
    m = torch.tensor([max(x, 1) for x in length], dtype=torch.float64, device="cuda")[:, None, None]
    rel = 2 * score + (32 + 6 * torch.log2(m) + m / 64) * U + split
    tol = rel * mean
    if t != F32:
        tol = tol + half(t) * (o.abs() + mean) + top * m * (2.0 ** -25 if t == F16 else 0)
        tol = tol + (2.0 ** -25 if t == F16 else 0)
    return tol, score[..., 0] + (rel[..., 0] + 4 * U) + 2 * U * lse.abs().nan_to_num(posinf=0, neginf=0)


def attention_case(seed, t, nh, nkv, hd, P, length, order="rows", spare=3, poison=True):
    """Pages in shuffled order; what no request may look at is NaN, and table
    entries behind a request's pages are no page."""
    g = gen(seed)
    held = [-(-max(m, 0) // P) for m in length]
    W = max(1, max(held))
    n_pages = sum(held) + spare
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(I32)
    table = torch.full((len(length), W), 2 ** 31 - 1, dtype=I32, device="cuda")
    shape = (n_pages, P, nkv, hd) if order == "rows" else (n_pages, nkv, P, hd)
    k, v = (torch.randn(*shape, generator=g, device="cuda").to(t) for _ in range(2))
    if order != "rows":
        k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = ids[at:at + h]
        at += h
        if poison and length[r] % P and length[r] > 0:
            for x in (k, v):
                x[int(table[r, h - 1]), length[r] % P:] = math.nan
    if poison:
        k[ids[at:].long()] = math.nan
        v[ids[at:].long()] = math.inf
    q = (1.5 * torch.randn(len(length), nh * hd, generator=g, device="cuda")).to(t)
    return q, k, v, table


def check_attention(qp, t, nh, nkv, hd, P, length, order="rows", seed=1, scale=None):
    q, k, v, table = attention_case(seed, t, nh, nkv, hd, P, length, order)
    lse = torch.full((len(length), nh), 7.0, device="cuda")
    status = status_word()
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev(length), nh, scale=scale, lse=lse, status=status)
    assert int(status) == 0
    want = attention_by_definition(q, k, v, table, length, nh, scale or 1 / math.sqrt(hd))
    tol, lse_tol = attention_tolerance(t, hd, length, want)
    close(o.view(-1, nh, hd), want[0], tol)
    close(lse, want[1], lse_tol)
    return o, lse


LENGTHS = [[1], [0], [2, 0, 1], [15, 16, 17, 63, 64, 65], [127, 128, 129, 0, 0, 1000, 3], [0, 0, 513]]


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(14, 2, 64), (28, 4, 128), (16, 8, 128), (4, 4, 64)])
@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("P,order", [(16, "rows"), (24, "heads")])
def test_paged_attention(qp, t, nh, nkv, hd, length, P, order):
    check_attention(qp, t, nh, nkv, hd, P, length, order, seed=len(length) + nh)


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(8, 1, 64), (9, 1, 128), (16, 1, 64), (17, 1, 128), (32, 1, 64), (64, 2, 64), (3, 1, 128)])
def test_paged_attention_head_groups(qp, t, nh, nkv, hd):
    check_attention(qp, t, nh, nkv, hd, 8, [5, 130, 0, 67], seed=nh)


@pytest.mark.parametrize("P", [1, 3, 64, 100, 1024])
def test_paged_attention_page_sizes(qp, P):
    check_attention(qp, F16, 12, 2, 128, P, [777, 1, 64, 2049], "heads", seed=P)


@pytest.mark.parametrize("t,length", [(BF16, [40001]), (F32, [9000, 1]), (F16, [131071])])
def test_paged_attention_long(qp, t, length):
    check_attention(qp, t, 14, 2, 64, 64, length)


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("nh,nkv", [(7, 1), (12, 2), (32, 2)])
@pytest.mark.parametrize("length", [[6000, 0, 2047], [30001]])
def test_paged_attention_long_wide_heads(qp, t, nh, nkv, length):
    check_attention(qp, t, nh, nkv, 128, 48, length, "heads")


def test_paged_attention_many_ragged_requests(qp):
    rng = random.Random(3)
    length = [rng.choice([0, 1, rng.randint(2, 300), rng.randint(1, 40)]) for _ in range(701)]
    check_attention(qp, BF16, 4, 2, 64, 16, length)


def test_paged_attention_scale_and_strides(qp):
    """Q as a slice of fused rows, output rows of a wider buffer, a table that is a slice; a scale of the caller's."""
    nh, nkv, hd, length = 4, 2, 64, [33, 70, 5]
    q, k, v, table = attention_case(9, BF16, nh, nkv, hd, 16, length)
    wide = torch.randn(3, nh * hd + 256, device="cuda").to(BF16)
    wide[:, 64:64 + nh * hd] = q
    out = torch.full((3, nh * hd + 64), 5.0, dtype=BF16, device="cuda")
    big = torch.full((3, 40), 2 ** 31 - 1, dtype=I32, device="cuda")
    big[:, 3:3 + table.shape[1]] = table
    cache = qp.PagedCache(k, v)
    qp.op_paged_attention(wide[:, 64:64 + nh * hd], cache, big[:, 3:], dev(length), nh, scale=0.31, out=out[:, :nh * hd])
    assert torch.equal(out[:, :nh * hd], qp.op_paged_attention(q, cache, table, dev(length), nh, scale=0.31))
    assert (out[:, nh * hd:] == 5).all()
    want = attention_by_definition(q, k, v, table, length, nh, 0.31)
    close(out[:, :nh * hd].view(3, nh, hd), want[0], attention_tolerance(BF16, hd, length, want)[0])


@pytest.mark.parametrize("t", [F32, BF16])
def test_paged_attention_rising_scores(qp, t):
    """Keys whose scores grow along the request: the running maximum moves at
    every unit, and the first keys' weights underflow."""
    nh, nkv, hd, m = 7, 1, 64, 1500
    q, k, v, table = attention_case(5, t, nh, nkv, hd, 16, [m], poison=False)
    q = q.abs().clamp(0.1, 2)
    flat = torch.linspace(-3, 3, table.shape[1] * 16, device="cuda")
    k[table[0].long()] = (flat.view(-1, 16, 1, 1) + 0.1 * k[table[0].long()].float()).to(t)
    lse = torch.empty(1, nh, device="cuda")
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh, lse=lse)
    want = attention_by_definition(q, k, v, table, [m], nh, 1 / math.sqrt(hd))
    tol, lse_tol = attention_tolerance(t, hd, [m], want)
    close(o.view(-1, nh, hd), want[0], tol)
    close(lse, want[1], lse_tol)


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_paged_attention_refuses_requests_on_the_device(qp, t):
    """Bad lengths and page ids: those requests' rows stay as they were, the
    others are what they are without them."""
    nh, nkv, hd, P = 14, 2, 64, 16
    length = [100, 5000, 64, 40, 900, 1]
    q, k, v, table = attention_case(2, t, nh, nkv, hd, P, length)
    cache = qp.PagedCache(k, v)
    cap = table.shape[1] * P
    good = qp.op_paged_attention(q, cache, table, dev(length), nh)
    for r, what in ((0, -1), (1, cap + 1), (3, -2 ** 31), (1, "page"), (0, "page"), (5, "page"), (1, "negative page"), (4, "last page")):
        ln, tb = list(length), table.clone()
        if what == "page":
            tb[r, 0] = k.shape[0]
        elif what == "negative page":
            tb[r, 150] = -1
        elif what == "last page":
            tb[r, -(-ln[r] // P) - 1] = 2 ** 31 - 1
        else:
            ln[r] = what
        out, lse = torch.full_like(q, 3.0), torch.full((len(ln), nh), 3.0, device="cuda")
        status = status_word()
        qp.op_paged_attention(q, cache, tb, dev(ln), nh, out=out, lse=lse, status=status)
        assert int(status) == -2, (r, what)
        assert (out[r] == 3).all() and (lse[r] == 3).all(), (r, what)
        rest = [i for i in range(len(ln)) if i != r]
        # other shares cut the same sums elsewhere: equal up to the two calls' roundings
        want = attention_by_definition(q, k, v, table, length, nh, 1 / math.sqrt(hd))
        tol, _ = attention_tolerance(t, hd, length, want)
        close(out[rest].view(-1, nh, hd), good[rest].view(-1, nh, hd), 2 * tol[rest])
        close(out[rest].view(-1, nh, hd), want[0][rest], tol[rest])


@pytest.mark.parametrize("t,nh,nkv,hd", [(BF16, 14, 2, 64), (F16, 16, 1, 128), (F32, 12, 2, 128)])
def test_paged_attention_refuses_a_long_request(qp, t, nh, nkv, hd):
    """A bad page in one of many shares: the mark goes through both levels of the
    join, and the next call with the same workspace is what it should be."""
    length, P = [20000, 77], 16
    q, k, v, table = attention_case(6, t, nh, nkv, hd, P, length)
    cache = qp.PagedCache(k, v)
    work = qp.op_paged_attention_workspace(cache, 2, nh)
    good = qp.op_paged_attention(q, cache, table, dev(length), nh, workspace=work)
    for page in (0, 600, 1249):
        bad = table.clone()
        bad[0, page] = -1
        out, status = torch.full_like(q, 3.0), status_word()
        qp.op_paged_attention(q, cache, bad, dev(length), nh, out=out, workspace=work, status=status)
        assert int(status) == -2 and (out[0] == 3).all() and torch.equal(out[1], good[1])
    assert torch.equal(good, qp.op_paged_attention(q, cache, table, dev(length), nh, workspace=work))
    assert int(work.buffer[:4096].sum()) == 0  # the counters


def test_workspaces_serve_calls_of_other_sizes(qp):
    """One workspace for calls of several shapes in turn: what one leaves behind
    does not reach the next."""
    nh, nkv, hd = 14, 2, 64
    cases = [attention_case(i, BF16, nh, nkv, hd, 16, length) + (length,) for i, length in enumerate(([5000], [3, 900, 0, 64], [1] * 40))]
    work = qp.op_paged_attention_workspace(qp.PagedCache(cases[0][1], cases[0][2]), 40, nh)
    g = gen(2)
    logits = [torch.randn(r, v, generator=g, device="cuda").to(t) for r, v, t in ((300, 20000, F32), (7, 9999, BF16), (1, 151936, F32), (1200, 600, F16))]
    lwork = max((qp.op_token_logprobs_workspace(x, 9) for x in logits), key=lambda w: w.nbytes)
    for _ in range(2):
        for q, k, v, table, length in cases:
            cache = qp.PagedCache(k, v)
            a = qp.op_paged_attention(q, cache, table, dev(length), nh, workspace=work)
            assert torch.equal(a, qp.op_paged_attention(q, cache, table, dev(length), nh))
        for x in logits:
            a, b = (qp.op_token_logprobs(x, None, 9, workspace=w) for w in (lwork, None))
            assert all(torch.equal(i, j) for i, j in zip(a[1:], b[1:]))


def test_paged_attention_shared_pages_and_repeats(qp):
    """Requests that share their first pages, and the same call twice: equal bits."""
    nh, nkv, hd, P = 12, 2, 128, 16
    q, k, v, table = attention_case(8, BF16, nh, nkv, hd, P, [200, 200, 200])
    table[1, :9] = table[0, :9]
    table[2] = table[0]
    cache = qp.PagedCache(k, v)
    a = qp.op_paged_attention(q, cache, table, dev([200, 200, 200]), nh)
    b = qp.op_paged_attention(q, cache, table, dev([200, 200, 200]), nh)
    assert torch.equal(a, b)
    want = attention_by_definition(q, k, v, table, [200] * 3, nh, 1 / math.sqrt(hd))
    close(a.view(-1, nh, hd), want[0], attention_tolerance(BF16, hd, [200] * 3, want)[0])


def test_paged_attention_infinite_values(qp):
    """An infinite V row that a request sees makes its dims infinite; one that it
    does not see changes nothing.  Scores of -inf weigh nothing."""
    nh, nkv, hd, P = 4, 2, 64, 16
    q, k, v, table = attention_case(3, BF16, nh, nkv, hd, P, [40, 40])
    cache = qp.PagedCache(k, v)
    base = qp.op_paged_attention(q, cache, table, dev([40, 40]), nh)
    v[int(table[0, 1]), 3, 0, 5] = math.inf
    o = qp.op_paged_attention(q, cache, table, dev([40, 40]), nh)
    assert (o[0].view(nh, hd)[:2, 5] == math.inf).all()
    o[0].view(nh, hd)[:2, 5] = base[0].view(nh, hd)[:2, 5]
    assert torch.equal(o, base)


# ------------------------------------------------------------------ log probabilities
def logprobs_by_definition(x, ids, k):
    x = x.double()
    top = x.amax(-1, keepdim=True)
    none = torch.isneginf(top)
    z = torch.where(none, 0.0, top)
    e = torch.exp(x - z)
    s = e.sum(-1, keepdim=True)
    logp = torch.where(none, -math.inf, (x - z) - torch.log(s))
    h = torch.where(none, 0.0, torch.log(s) - torch.where(e > 0, e * (x - z), 0.0).sum(-1, keepdim=True) / s)[:, 0]
    # equal values by ascending id, NaN above +inf
    order = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :k]
    return logp.gather(1, ids.long()[:, None])[:, 0], h, order.to(I32), logp.gather(1, order)


def logprobs_tolerance(x, logp):
    """ln s: a thread adds up to V / 256 + 1 terms of at most 3 ulp each, 16 more
    adds join them; y - z and its parts 3 U of their size; log2 2 ulp."""
    V = x.shape[1]
    return (V / 256 + 17 + 6 + 4) * U + 4 * U * logp.abs().nan_to_num(posinf=0, neginf=0)


def check_logprobs(qp, x, ids, k):
    rows = x.shape[0]
    status = status_word()
    logprob, entropy, top_ids, top_logprobs = qp.op_token_logprobs(x, ids, k, status=status)
    assert int(status) == 0
    lp, h, order, tl = logprobs_by_definition(x, ids, k)
    assert torch.equal(top_ids, order)
    close(logprob, lp, logprobs_tolerance(x, lp))
    close(top_logprobs, tl, logprobs_tolerance(x, tl))
    # t / s: the same relative errors on a mean of |y - z|, which is at most H / ln 2 + log2 V
    close(entropy, h, 2 * logprobs_tolerance(x, h + math.log(max(2, x.shape[1]))) * (1 + h.abs() + math.log(max(2, x.shape[1]))))
    assert rows == logprob.shape[0]


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("rows,V,extra,k", [(1, 1, 0, 1), (3, 2, 1, 2), (2, 31, 3, 31), (5, 33, 0, 32), (7, 257, 1, 5), (2, 1000, 7, 32),
                                            (3, 4096, 0, 20), (4, 4097, 1, 1), (2, 20001, 3, 8), (1, 151936, 0, 5), (33, 151936, 0, 0),
                                            (9, 150001, 5, 32)])
def test_token_logprobs(qp, t, rows, V, extra, k):
    g = gen(V + rows)
    x = (3 * torch.randn(rows, V + extra, generator=g, device="cuda")).to(t)[:, :V]
    ids = torch.randint(0, V, (rows,), generator=g, device="cuda").to(I32)
    check_logprobs(qp, x, ids, k)


@pytest.mark.parametrize("rows", [600, 5000])
def test_token_logprobs_many_rows(qp, rows):
    g = gen(rows)
    x = 2 * torch.randn(rows, 5001, generator=g, device="cuda")
    check_logprobs(qp, x, torch.randint(0, 5001, (rows,), generator=g, device="cuda").to(I32), 7)


@pytest.mark.parametrize("kind", ["equal", "two levels", "rising", "falling", "one left", "two left", "none left", "huge", "tiny", "peak",
                                  "zeros of both signs", "lowest"])
@pytest.mark.parametrize("V,k", [(5000, 20), (151936, 32), (40, 32)])
def test_token_logprobs_hard_rows(qp, kind, V, k):
    g = gen(V)
    rows = 3
    x = torch.randn(rows, V, generator=g, device="cuda")
    if kind == "equal":
        x.fill_(1.25)
    elif kind == "two levels":
        x = (x > 1).float()
    elif kind == "rising":
        x = torch.linspace(-40, 40, V, device="cuda").repeat(rows, 1)
    elif kind == "falling":
        x = torch.linspace(40, -40, V, device="cuda").repeat(rows, 1)
    elif kind == "one left":
        x.fill_(-math.inf)
        x[:, V - 1] = -3.0
    elif kind == "two left":
        x.fill_(-math.inf)
        x[:, 0], x[:, V // 2] = 2.0, 2.0
    elif kind == "none left":
        x[1].fill_(-math.inf)
    elif kind == "huge":
        x *= 1e30
    elif kind == "tiny":
        x *= 1e-30
    elif kind == "peak":
        x[:, 7] = 60.0
    elif kind == "zeros of both signs":
        x = torch.where(x > 0, 0.0, -0.0)
    elif kind == "lowest":
        x = torch.where(x > 1, x, torch.finfo(F32).min)
    ids = torch.tensor([0, V - 1, V // 2], dtype=I32, device="cuda")
    check_logprobs(qp, x, ids, k)


@pytest.mark.parametrize("t", [F32, F16])
@pytest.mark.parametrize("kind", ["random", "side by side", "few levels", "two left", "none left"])
@pytest.mark.parametrize("k", [1, 9, 32])
def test_token_logprobs_wide_vocabularies(qp, t, kind, k):
    """Chunk maxima beyond the 512 that a join holds in registers; large values that share chunks."""
    g = gen(k)
    for V in (262143, 262145, 400003):
        x = torch.randn(2, V, generator=g, device="cuda")
        if kind == "side by side":  # one chunk and a half hold everything large, more than fits the list
            x[:, V - 800:] = 20 + x[:, V - 800:]
        elif kind == "few levels":
            x = (4 * x).round() / 4
        elif kind == "two left":
            x[:, 2:V - 1] = -math.inf
        elif kind == "none left":
            x[0].fill_(-math.inf)
        x = x.to(t)
        check_logprobs(qp, x, dev([0, V - 1]), k)


@pytest.mark.parametrize("V", [151936, 262145, 300001])
def test_token_logprobs_many_whole_rows(qp, V):
    """More rows than the GPU holds CTAs twice: every row is one CTA's, with its chunk maxima in shared memory or, past
    512 chunks, in the workspace."""
    rows = 2 * 4 * torch.cuda.get_device_properties(0).multi_processor_count + 7
    x = torch.randn(rows, V, generator=gen(V), device="cuda", dtype=F16)
    x[3].fill_(-math.inf)
    ids = (torch.arange(rows, device="cuda") * 37 % V).to(I32)
    status = status_word()
    got = qp.op_token_logprobs(x, ids, 9, status=status)
    assert int(status) == 0
    some = [0, 3, 4, rows // 2, rows - 1]
    for r in some:
        lp, h, order, tl = logprobs_by_definition(x[r:r + 1], ids[r:r + 1], 9)
        assert torch.equal(got[2][r], order[0])
        close(got[0][r:r + 1], lp, logprobs_tolerance(x, lp))
        close(got[3][r], tl[0], logprobs_tolerance(x, tl[0]))
        close(got[1][r:r + 1], h, 2 * logprobs_tolerance(x, h + math.log(V)) * (1 + h.abs() + math.log(V)))
    again = qp.op_token_logprobs(x, ids, 9, status=status)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


def test_token_logprobs_nan_and_infinity(qp):
    x = torch.randn(4, 3000, device="cuda")
    x[0, 0], x[0, 2999] = math.nan, math.inf
    x[1, 5], x[1, 9] = math.inf, math.inf
    x[2, 1:2000] = math.nan
    logprob, entropy, ids, lps = qp.op_token_logprobs(x, dev([3, 3, 3, 3]), 5)
    assert torch.isnan(logprob[:3]).all() and torch.isnan(entropy[:3]).all() and torch.isnan(lps[:3]).all()
    assert ids[0, :2].tolist() == [0, 2999] and ids[1, :2].tolist() == [5, 9] and ids[2].tolist() == [1, 2, 3, 4, 5]
    assert torch.isfinite(logprob[3]) and torch.isfinite(lps[3]).all()


def test_token_logprobs_padding_and_refused_rows(qp):
    x = torch.randn(5, 777, device="cuda")
    out = (torch.full((5,), 3.0, device="cuda"), torch.full((5,), 3.0, device="cuda"), torch.full((5, 4), 3, dtype=I32, device="cuda"),
           torch.full((5, 4), 3.0, device="cuda"))
    status = status_word()
    qp.op_token_logprobs(x, dev([5, -1, 776, -2 ** 31, 0]), 4, out=out, status=status)
    assert int(status) == 0
    for y in out:
        assert (y[[1, 3]] == 3).all() and not (y[[0, 2, 4]] == 3).all()
    want = logprobs_by_definition(x, dev([5, 0, 776, 0, 0]), 4)
    assert torch.equal(out[2][[0, 2, 4]], want[2][[0, 2, 4]])
    qp.op_token_logprobs(x, dev([5, 777, 776, 2 ** 31 - 1, 0]), 4, out=tuple(y.fill_(3) for y in out), status=status)
    assert int(status) == -3
    for y in out:
        assert (y[[1, 3]] == 3).all()
    assert torch.equal(out[2][[0, 2, 4]], want[2][[0, 2, 4]])
    # without ids every row is scored, and there is no log probability of a token
    logprob, entropy, ids, lps = qp.op_token_logprobs(x, None, 4)
    assert logprob is None and torch.equal(ids, want[2]) and torch.isfinite(entropy).all() and torch.isfinite(lps).all()


# ------------------------------------------------------------------ offsets past 32 bits
def test_offsets_past_32_bits(qp):
    """Pages 2^31 elements apart, logits rows 2^30 apart."""
    nh, nkv, hd, P = 4, 2, 64, 16
    far = 2 ** 31 + 64
    big = torch.empty(2 * far + P * nkv * hd, dtype=BF16, device="cuda")
    k = big.as_strided((3, P, nkv, hd), (far, nkv * hd, hd, 1))
    v = torch.empty_like(big).as_strided(k.shape, k.stride())
    g = gen(1)
    k.copy_(torch.randn(3, P, nkv, hd, generator=g, device="cuda"))
    v.copy_(torch.randn(3, P, nkv, hd, generator=g, device="cuda"))
    cache, table = qp.PagedCache(k, v), dev([[2, 0, 1]])
    q = torch.randn(1, nh * hd, generator=g, device="cuda").to(BF16)
    o = qp.op_paged_attention(q, cache, table, dev([45]), nh)
    want = attention_by_definition(q, k, v, table, [45], nh, 1 / 8)
    close(o.view(1, nh, hd), want[0], attention_tolerance(BF16, hd, [45], want)[0])
    qkv = torch.randn(2, 8 * hd, generator=g, device="cuda").to(BF16)
    qp.op_rope_paged_store(qkv, qp.RopeTable(hd), dev([3, 4]), dev([2 * P + 5, P + 1]), cache, nh)
    assert torch.equal(v[2, 5].flatten(), qkv[0, 6 * hd:]) and torch.equal(v[1, 1].flatten(), qkv[1, 6 * hd:])
    del big, k, v, cache
    x = torch.empty(2 ** 31 + 2 ** 30 + 4096, dtype=F16, device="cuda").as_strided((4, 4096), (2 ** 30, 1))
    x.copy_(torch.randn(4, 4096, generator=g, device="cuda"))
    check_logprobs(qp, x, dev([1, 2, 3, 4095]), 6)


# ------------------------------------------------------------------ streams, graphs, a run together
def test_streams_and_captured_graphs(qp):
    """Two graphs captured from the same operators on one side stream, replayed
    with other inputs, and two calls at once on two streams: each has what a
    plain call gives."""
    nh, nkv, hd, P = 14, 2, 64, 16
    length = [300, 1, 0, 777]
    q, k, v, table = attention_case(4, BF16, nh, nkv, hd, P, length)
    cache, ln = qp.PagedCache(k, v), dev(length)
    x = torch.randn(4, 30000, device="cuda")
    ids = dev([1, 2, 3, 4])
    side = torch.cuda.Stream()
    graphs = []
    for i in range(2):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            qp.op_paged_attention(q, cache, table, ln, nh)
            qp.op_token_logprobs(x, ids, 5)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o = qp.op_paged_attention(q, cache, table, ln, nh)
            lp = qp.op_token_logprobs(x, ids, 5)
        graphs.append((graph, o, lp))
    q.copy_(torch.randn(4, nh * hd, device="cuda"))
    ln.copy_(dev([299, 0, 0, 500]))
    x.mul_(0.5)
    torch.cuda.synchronize()
    for graph, *_ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = qp.op_paged_attention(q, cache, table, ln, nh)
    want_lp = qp.op_token_logprobs(x, ids, 5)
    for _, o, lp in graphs:
        assert torch.equal(o, want)
        assert all(torch.equal(a, b) for a, b in zip(lp, want_lp))
    other = torch.cuda.Stream()
    for s in (side, other):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(20):
        for s in (side, other):
            with torch.cuda.stream(s):
                got.append((qp.op_paged_attention(q, cache, table, ln, nh), qp.op_token_logprobs(x, ids, 5)))
    torch.cuda.synchronize()
    for o, lp in got:
        assert torch.equal(o, want) and all(torch.equal(a, b) for a, b in zip(lp, want_lp))


@pytest.mark.parametrize("captured", [False, True])
def test_a_batch_served_step_by_step(qp, captured):
    """Requests come, grow by prompts and single tokens, are rolled back and end;
    every step runs page tables, RoPE with the store, attention of each
    request's last token and log probabilities, against a dense 64-bit cache
    kept per request.  With `captured` one graph of the step is replayed."""
    nh, nkv, hd, P, n, W, V = 4, 2, 64, 16, 5, 8, 999
    width, max_tokens, n_pages = (nh + 2 * nkv) * hd, 160, 24
    rng = random.Random(11)
    g = gen(11)
    k, v = (torch.full((n_pages, P, nkv, hd), math.nan, device="cuda") for _ in range(2))
    cache, rope = qp.PagedCache(k, v), qp.RopeTable(hd, 32, 1e4, "interleaved", "linear", 2.0)
    ln, target = torch.zeros(n, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda")
    table = torch.full((n, W), -1, dtype=I32, device="cuda")
    free, n_free = torch.arange(n_pages, dtype=I32, device="cuda"), dev([n_pages])
    qkv, bias = torch.zeros(max_tokens, width, device="cuda"), torch.randn(width, generator=g, device="cuda")
    head = torch.randn(nh * hd, V, generator=g, device="cuda") / 8
    ids, status = torch.zeros(n, dtype=I32, device="cuda"), status_word()

    def step():
        start, pos, slot, _ = qp.op_page_tables(ln, target, P, table, free, n_free, n_pages, max_tokens,
                                                out=(s_start, s_pos, s_slot, n_free), status=status)
        q = qp.op_rope_paged_store(qkv, rope, pos, slot, cache, nh, bias=bias, out=s_q, status=status)
        last = q[(start[1:].long() - 1).clamp(min=0)]
        o = qp.op_paged_attention(last, cache, table, target, nh, status=status)
        x = o @ head
        ln.copy_(target)
        return last, o, x, qp.op_token_logprobs(x, ids, 3, status=status)

    s_start, s_pos, s_slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (n + 1, max_tokens, max_tokens))
    s_q = torch.zeros(max_tokens, nh * hd, device="cuda")
    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # lengths are all 0 and so are the targets: nothing moves
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = step()
    f, scale = rope_frequencies(32, 1e4, "linear", 2.0, 0)
    dense = [(torch.zeros(0, nkv, hd, dtype=torch.float64, device="cuda"),) * 2 for _ in range(n)]
    have = [0] * n
    for i in range(12):
        want = []
        for r in range(n):
            kind = rng.choice(["prompt", "one", "one", "one", "back", "over"])
            want.append({"prompt": have[r] + rng.randint(1, 30), "one": have[r] + 1, "back": max(0, have[r] - rng.randint(0, 20)), "over": 0}[kind])
            want[r] = min(want[r], 64)
        new = [max(0, b - a) for a, b in zip(have, want)]
        qkv.fill_(math.nan)
        qkv[:sum(new)] = torch.randn(sum(new), width, generator=g, device="cuda")
        target.copy_(dev(want))
        ids.copy_(torch.randint(0, V, (n,), generator=g, device="cuda"))
        if captured:
            graph.replay()
        else:
            result = step()
        last, o, x, lp = result
        assert int(status) == 0
        pages = [p for r in range(n) for p in table[r, :-(-want[r] // P)].tolist()]
        assert sorted(pages + free[:int(n_free)].tolist()) == list(range(n_pages))  # each page in one place
        at = 0
        for r in range(n):
            pos = torch.arange(have[r], have[r] + new[r], device="cuda")
            y, _ = rope_by_formula(qkv[at:at + new[r]], nh, nkv, hd, pos, f, scale, "interleaved", bias)
            at += new[r]
            kk, vv = (torch.cat([a[:min(have[r], want[r])], b]) for a, b in zip(dense[r], (y[:, nh:nh + nkv], y[:, nh + nkv:])))
            dense[r] = (kk, vv)
            assert kk.shape[0] == want[r]
            if want[r]:
                s = torch.einsum("hgd,jhd->hgj", last[r].double().view(nkv, nh // nkv, hd), kk) / math.sqrt(hd)
                exact = torch.einsum("hgj,jhd->hgd", torch.softmax(s, -1), vv).flatten()
                # the stored rows are off by ROPE_F32 of at most |x| + |bias| <= 12, scores and weights with them
                size = float(last[r].double().abs().sum() / nh / math.sqrt(hd)) * 12 * ROPE_F32 * 4
                close(o[r], exact, 12 * (2 * size + ROPE_F32 + 2.0 ** -16))
            else:
                assert (o[r] == 0).all()
        want_lp = logprobs_by_definition(x, ids, 3)
        assert torch.equal(lp[2], want_lp[2])
        close(lp[0], want_lp[0], logprobs_tolerance(x, want_lp[0]))
        have = want


def test_logits_rows_of_a_model_are_scored(qp):
    """The rows of minfer_prefill_device_n go straight into op_token_logprobs."""
    import synth
    from helpers import gpu_model
    cfg, w = synth.TINY, synth.WORKLOADS["tiny-32"]
    m = gpu_model(cfg)
    kv = m.kv(w.n_ctx)
    ids, pos = dev(w.ids().tolist()), dev(w.positions().tolist())
    logits = torch.empty(32, cfg.n_vocab, device="cuda")
    torch.cuda.synchronize()
    assert m.prefill_device_n(kv, ids.data_ptr(), pos.data_ptr(), 32, 32, logits.data_ptr()) == 0
    assert m.sync_status() == 0
    check_logprobs(qp, logits, torch.cat([ids[1:], ids[:1]]), 5)


def test_outputs_of_another_layout_are_refused(qp):
    """An output with as many elements as wanted, laid out otherwise, is refused before any launch."""
    cache = qp.PagedCache(torch.zeros(4, 16, 2, 64, device="cuda"), torch.zeros(4, 16, 2, 64, device="cuda"))
    q, length, table = torch.zeros(3, 256, device="cuda"), dev([1, 1, 1]), dev([[0], [1], [2]])
    with pytest.raises(qp.MinferError, match="lse"):
        qp.op_paged_attention(q, cache, table, length, 4, lse=torch.zeros(4, 3, device="cuda"))
    with pytest.raises(qp.MinferError, match="out"):
        qp.op_paged_attention(q, cache, table, length, 4, out=torch.zeros(256, 3, device="cuda"))
    x, ids = torch.zeros(3, 50, device="cuda"), dev([1, 2, 3])
    out = [torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda"), torch.zeros(3, 2, dtype=I32, device="cuda"),
           torch.zeros(3, 2, device="cuda")]
    qp.op_token_logprobs(x, ids, 2, out=tuple(out))
    for i in (2, 3):
        wrong = list(out)
        wrong[i] = torch.zeros(2, 3, dtype=out[i].dtype, device="cuda")
        with pytest.raises(qp.MinferError, match="top"):
            qp.op_token_logprobs(x, ids, 2, out=tuple(wrong))
    with pytest.raises(qp.MinferError, match="k: -1"):
        qp.op_token_logprobs(x, ids, -1)
