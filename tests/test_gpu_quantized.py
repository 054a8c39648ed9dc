"""The operators of a Q8_0 paged cache on the GPU against plain 64-bit
implementations: RoPE with the quantizing store, rows read back, attention of one
token per request, and a run of them together."""
import math
import os
import random
import re

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_batch import (BF16, F16, F32, I32, ROPE_F32, U, attention_by_definition, close, dev, gen, half,  # noqa: E402
                            rope_by_formula, rope_frequencies, status_word)


@pytest.fixture(scope="module")
def qp():
    import quantized_transformer_prefill_gb300 as qp
    qp.lib()
    return qp


def pool(g, n_pages, P, nkv, hd, order="rows", amp=0.01):
    """Random codes (any int8) and scales, as k, v, k_scale, v_scale."""
    shape = (n_pages, P, nkv) if order == "rows" else (n_pages, nkv, P)
    view = (lambda x: x) if order == "rows" else (lambda x: x.permute(0, 2, 1, 3))
    k, v = (view(torch.randint(-128, 128, (*shape, hd), generator=g, device="cuda", dtype=torch.int8)) for _ in range(2))
    ks, vs = (view((amp * (0.2 + torch.rand(*shape, hd // 32, generator=g, device="cuda"))).half()) for _ in range(2))
    return k, v, ks, vs


def values(codes, scales):
    """What the blocks stand for, exact in f32."""
    return (codes.float().unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def codec(x):
    """Codes and scales of f32 rows [..., hd], every step one f32 rounding (on the host)."""
    b = x.float().cpu().unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / torch.tensor(127.0)
    y = b * torch.where(d > 0, 1 / d, 0.0)
    code = torch.copysign(torch.floor(y.double().abs() + 0.5), y.double()).clamp(-127, 127)
    return code.flatten(-2).to(torch.int8), d[..., 0].half()


# ------------------------------------------------------------------ RoPE with the quantizing store
STORE_CASES = [
    # nh, nkv, hd, src, to, page, style, rot, scaling, norm, bias
    (14, 2, 64, BF16, BF16, 16, "half", 64, "none", False, True),
    (14, 2, 64, F32, F32, 16, "interleaved", 64, "none", False, True),
    (12, 2, 128, F32, BF16, 1, "half", 128, "yarn", False, True),
    (16, 8, 128, F16, F16, 24, "interleaved", 64, "linear", True, False),
    (16, 8, 128, F32, F32, 32, "half", 24, "ntk", True, False),
    (4, 2, 64, F32, F16, 128, "half", 6, "none", True, True),
    (5, 1, 128, BF16, BF16, 16, "half", 90, "linear", True, True),
    (160, 32, 128, F32, F16, 16, "interleaved", 90, "yarn", False, True),
    (3, 3, 64, F16, F16, 16, "half", 20, "none", True, True),
    (1, 1, 64, BF16, BF16, 3, "half", 64, "none", False, False),
]


@pytest.mark.parametrize("nh,nkv,hd,src,to,P,style,rot,scaling,norm,bias", STORE_CASES)
@pytest.mark.parametrize("n,order", [(1, "rows"), (37, "heads"), (700, "rows")])
def test_store(qp, nh, nkv, hd, src, to, P, style, rot, scaling, norm, bias, n, order):
    g = gen(n + hd)
    width = (nh + 2 * nkv) * hd
    qkv = torch.randn(n, width + 64, generator=g, device="cuda").to(src)[:, :width]
    b = torch.randn(width, generator=g, device="cuda") if bias else None
    norms = tuple(1 + 0.2 * torch.randn(hd, generator=g, device="cuda") for _ in range(2)) if norm else None
    pages = -(-n // P) + 2
    before = pool(g, pages, P, nkv, hd, order)
    after = tuple(x.clone(memory_format=torch.preserve_format) for x in before)
    pos = torch.randint(0, 2 ** 31 - 1, (n,), generator=g, device="cuda").to(I32)
    slot = torch.randperm(pages * P, generator=g, device="cuda")[:n].to(I32)
    pad = torch.zeros(n, dtype=torch.bool, device="cuda")
    pad[n // 3::5] = n > 1
    pos[pad], slot[pad] = -1, -1
    qkv[pad] = math.nan  # what a padding row holds is not looked at
    out = torch.full((n, nh * hd + 8), 7.0, dtype=to, device="cuda")[:, :nh * hd]
    ctx, factor, theta = 4096, 1.0 if scaling == "none" else 4.0, 1e6
    status = status_word()
    qp.op_rope_paged_store_q8(qkv, qp.RopeTable(hd, rot, theta, style, scaling, factor, ctx), pos, slot, qp.PagedCacheQ8(*after), nh, bias=b,
                              q_norm=norms and norms[0], k_norm=norms and norms[1], eps=1e-6, out=out, status=status)
    assert int(status) == 0
    f, scale = rope_frequencies(rot, theta, scaling, factor, ctx)
    live = ~pad
    want, bound = rope_by_formula(qkv[live], nh, nkv, hd, pos[live], f, scale, style, b, norms)
    err = (ROPE_F32 + 2.0 ** -21) * bound  # of the f32 values that are rounded to Q's type or quantized
    close(out[live].view(-1, nh, hd), want[:, :nh],
          half(to) * want[:, :nh].abs() + err[:, :nh] + torch.finfo(to).smallest_normal * half(to) * 2)
    at = slot[live].long()
    for i, codes, scales in ((0, after[0], after[2]), (1, after[1], after[3])):
        part = slice(nh + i * nkv, nh + (i + 1) * nkv)
        x, e = (y[:, part].unflatten(-1, (-1, 32)) for y in (want, err))
        top, etop = x.abs().amax(-1, keepdim=True), e.amax(-1, keepdim=True)
        d = top / 127
        # the scale: the maximum's error, the division's rounding, and f16's
        close(scales[at // P, at % P], d[..., 0], (etop / 127 + 2.0 ** -11 * (d + etop) + 2.0 ** -23 * d + 2.0 ** -25)[..., 0])
        # the code: that of the exact value, but next to a border between two codes (the value's error and the maximum's
        # share of it in steps, and three roundings of a number up to 127)
        y = x / d
        want_code = torch.copysign(torch.floor(y.abs() + 0.5), y)
        off = (codes[at // P, at % P].double().unflatten(-1, (-1, 32)) - want_code).abs()
        near = ((y.abs() - y.abs().floor()) - 0.5).abs() <= (e + etop) / d * 1.01 + 3 * 127 * U
        assert (off <= near.double()).all(), float(off.max())
        if not norm and not bias and i == 1 and src == F32:  # V's values are what they were: every bit
            c, s = codec(qkv[live].view(-1, nh + 2 * nkv, hd)[:, part])
            assert torch.equal(codes[at // P, at % P].cpu(), c) and torch.equal(scales[at // P, at % P].cpu(), s)
    # nothing else is touched
    assert (out[pad] == 7).all()
    for x, y in zip(after, before):
        x[at // P, at % P] = y[at // P, at % P]
        assert torch.equal(x, y)


def test_stored_blocks_are_those_of_the_activations(qp):
    """V without a bias gets the bits of op_quantize, the codec of the matmul inputs: large and tiny blocks, ties, zeros."""
    n, hd = 64, 128
    g = gen(5)
    x = torch.randn(n, hd, generator=g, device="cuda") * torch.logspace(-12, 6, n, device="cuda")[:, None]
    x[3] = 0
    x[4, :32] = torch.arange(32, device="cuda") * 0.5 - 4
    x[4, 0] = 127.0  # a scale of 1: halves are ties
    qkv = torch.cat([torch.zeros(n, 2 * hd, device="cuda"), x], 1)
    k, v, ks, vs = (t.zero_() for t in pool(g, 4, 16, 1, hd))
    qp.op_rope_paged_store_q8(qkv, qp.RopeTable(hd), dev([0] * n), dev(list(range(n))), qp.PagedCacheQ8(k, v, ks, vs), 1)
    codes, bits = qp.op_quantize(x)
    assert torch.equal(v.view(n, hd), codes) and torch.equal(vs.view(n, 4).view(torch.int16), bits.view(torch.int16))
    assert not k.any() and not ks.any()
    c, s = codec(x)
    assert torch.equal(codes.cpu(), c) and torch.equal(vs.view(n, 4).cpu(), s)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 8.4e6, -3e38])
@pytest.mark.parametrize("src", [F32, BF16])
def test_blocks_without_a_scale_read_back_as_nan(qp, bad, src):
    n, nh, nkv, hd = 3, 2, 2, 64
    g = gen(9)
    qkv = torch.randn(n, 6 * hd, generator=g, device="cuda").to(src)
    qkv[1, 5 * hd + 40] = bad  # V, head 1, block 1
    cache = qp.PagedCacheQ8(*pool(g, 2, 4, nkv, hd))
    q = qp.op_rope_paged_store_q8(qkv, qp.RopeTable(hd), dev([1, 2, 3]), dev([0, 5, 2]), cache, nh)
    k, v = qp.op_paged_read_q8(cache, dev([0, 5, 2]))
    hit = torch.zeros(n, 2 * hd, dtype=torch.bool, device="cuda")
    hit[1, hd + 32:] = True
    assert torch.equal(torch.isnan(v), hit) and torch.isfinite(k).all() and torch.isfinite(q).all()
    close(v[~hit], qkv[:, 4 * hd:][~hit], 5 / 127 * 0.51)


def test_store_refuses_rows_on_the_device(qp):
    """A slot past the pool or a negative position: that row is not written."""
    n, nh, nkv, hd, P = 4, 4, 2, 64, 4
    g = gen(2)
    qkv = torch.randn(n, 8 * hd, generator=g, device="cuda")
    for pos, slot in (([0, 1, 2, 3], [0, 8, 2, 3]), ([0, -1, 2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 2 ** 31 - 1, 2, 3])):
        before = pool(g, 2, P, nkv, hd)
        after = tuple(x.clone() for x in before)
        out = torch.full((n, nh * hd), 3.0, device="cuda")
        status = status_word()
        qp.op_rope_paged_store_q8(qkv, qp.RopeTable(hd), dev(pos), dev(slot), qp.PagedCacheQ8(*after), nh, out=out, status=status)
        assert int(status) == -2
        assert (out[1] == 3).all() and not (out[[0, 2, 3]] == 3).any()
        kept = torch.tensor([r for r in range(2 * P) if r not in (0, 2, 3)], device="cuda")
        for x, y in zip(after, before):
            assert torch.equal(x.reshape(2 * P, -1)[kept], y.reshape(2 * P, -1)[kept])


# ------------------------------------------------------------------ rows read back
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("n,P,nkv,hd,order", [(1, 16, 2, 64, "rows"), (513, 16, 2, 64, "heads"), (1000, 24, 3, 128, "rows"), (77, 1, 8, 128, "heads"),
                                              (5, 7, 70, 128, "rows"), (3001, 64, 1, 64, "rows")])
def test_read(qp, t, n, P, nkv, hd, order):
    g = gen(n)
    pages = -(-n // P) + 1
    k, v, ks, vs = pool(g, pages, P, nkv, hd, order)
    slot = torch.randint(0, pages * P, (n,), generator=g, device="cuda").to(I32)  # some of them twice
    pad = torch.zeros(n, dtype=torch.bool, device="cuda")
    pad[n // 3::5] = n > 1
    slot[pad] = -1
    cache, status = qp.PagedCacheQ8(k, v, ks, vs), status_word()
    at = slot.long().clamp(min=0)
    want = [values(c[at // P, at % P], s[at // P, at % P]).flatten(1).to(t) for c, s in ((k, ks), (v, vs))]
    new = lambda: torch.full((n, nkv * hd + 8), 7.0, dtype=t, device="cuda")[:, :nkv * hd]  # noqa: E731
    a, b, one, two = new(), new(), new(), new()
    qp.op_paged_read_q8(cache, slot, out=(a, b), status=status)
    qp.op_paged_read_q8(cache, slot, out=(one, None), status=status)
    qp.op_paged_read_q8(cache, slot, out=(None, two), status=status)
    fresh = qp.op_paged_read_q8(cache, slot, dtype=t, status=status)
    assert int(status) == 0
    for got, w in ((a, want[0]), (b, want[1]), (one, want[0]), (two, want[1])):
        assert torch.equal(got[~pad], w[~pad]) and (got[pad] == 7).all()
    for got, w in zip(fresh, want):
        assert torch.equal(got[~pad], w[~pad]) and (got[pad] == 0).all()


def test_read_refuses_rows_on_the_device(qp):
    g = gen(1)
    parts = pool(g, 2, 4, 2, 64)
    cache = qp.PagedCacheQ8(*parts)
    for bad in (8, 2 ** 31 - 1):
        status = status_word()
        out = tuple(torch.full((3, 128), 7.0, device="cuda") for _ in range(2))
        qp.op_paged_read_q8(cache, dev([1, bad, 7]), out=out, status=status)
        assert int(status) == -2
        for got, c, s in zip(out, parts[:2], parts[2:]):
            assert (got[1] == 7).all() and torch.equal(got[[0, 2]], values(c, s).view(8, 128)[[1, 7]])


# ------------------------------------------------------------------ attention
def q8_tolerance(t, hd, length, want):
    """attention_by_definition's terms.  Score error: the MMA sums of a block cut off (2^-23 of the partial sum, hd / 8 + 2 of
    them over the row with the blocks' multiply-adds); f32 queries in two f16 numbers lose 2^-22, bf16 ones 2^-39 of the
    largest; the scaled score's rounding and the exponential's 2 ulp come on top.  Each weight's relative error is the score
    error twice (its own and the sum's); times its scale it is rounded (U) and split: two f16 numbers leave 2^-22, 4 U as
    counted for f32, less than the 2^-18 counted for 16-bit results; sums of up to 64 + units adds, the tensor core's (2 U) two
    or three a unit of 64 keys for 16-bit results."""
    o, lse, mean, size, top = want
    score = size * ((hd // 8 + 2) * 2.0 ** -23 + 2.0 ** -22 + 4 * U) + 8 * U
    m = torch.tensor([max(x, 1) for x in length], dtype=torch.float64, device="cuda")[:, None, None]
    rel = 2 * score + (32 + 6 * torch.log2(m) + m / 64 * (1 if t == F32 else 4)) * U + (4 * U if t == F32 else 2.0 ** -18 + U)
    tol = rel * mean
    if t != F32:
        tol = tol + half(t) * (o.abs() + tol) + (2.0 ** -25 if t == F16 else 0)
    return tol, score[..., 0] + (rel[..., 0] + 4 * U) + 2 * U * lse.abs().nan_to_num(posinf=0, neginf=0)


def q8_case(seed, t, nh, nkv, hd, P, length, order="rows", spare=3, amp=0.02):
    """Pages in shuffled order; the scales of what no request may look at are NaN, and table entries behind a request's pages
    are no page."""
    g = gen(seed)
    held = [-(-max(m, 0) // P) for m in length]
    W = max(1, max(held))
    n_pages = sum(held) + spare
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(I32)
    table = torch.full((len(length), W), 2 ** 31 - 1, dtype=I32, device="cuda")
    parts = pool(g, n_pages, P, nkv, hd, order, amp)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = ids[at:at + h]
        at += h
        if length[r] % P and length[r] > 0:
            for x in parts[2:]:
                x[int(table[r, h - 1]), length[r] % P:] = math.nan
    for x in parts[2:]:
        x[ids[at:].long()] = math.inf
    q = (1.5 * torch.randn(len(length), nh * hd, generator=g, device="cuda")).to(t)
    return q, parts, table


def check_q8(qp, t, nh, nkv, hd, P, length, order="rows", seed=1, scale=None, amp=0.02, change=None):
    q, parts, table = q8_case(seed, t, nh, nkv, hd, P, length, order, amp=amp)
    if change:
        change(q, parts, table)
    lse = torch.full((len(length), nh), 7.0, device="cuda")
    status = status_word()
    o = qp.op_paged_attention_q8(q, qp.PagedCacheQ8(*parts), table, dev(length), nh, scale=scale, lse=lse, status=status)
    assert int(status) == 0 and o.dtype == t
    want = attention_by_definition(q, values(parts[0], parts[2]), values(parts[1], parts[3]), table, length, nh, scale or 1 / math.sqrt(hd))
    tol, lse_tol = q8_tolerance(t, hd, length, want)
    exact = want[0]
    if t == F16:  # 65520, half a step past f16's largest number, and more round to infinity
        exact = torch.where(exact.abs() - tol >= 65520, torch.copysign(torch.full_like(exact, math.inf), exact), exact)
    close(o.view(-1, nh, hd), exact, tol)
    close(lse, want[1], lse_tol)
    return o, lse


LENGTHS = [[1], [0], [2, 0, 1], [15, 16, 17, 63, 64, 65], [127, 128, 129, 0, 0, 1000, 3], [0, 0, 513]]


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(14, 2, 64), (28, 4, 128), (16, 8, 128), (4, 4, 64)])
@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("P,order", [(16, "rows"), (24, "heads")])
def test_attention(qp, t, nh, nkv, hd, length, P, order):
    check_q8(qp, t, nh, nkv, hd, P, length, order)


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(8, 1, 64), (9, 1, 128), (16, 1, 64), (17, 1, 128), (32, 1, 64), (64, 2, 64), (3, 1, 128)])
def test_attention_head_groups(qp, t, nh, nkv, hd):
    check_q8(qp, t, nh, nkv, hd, 16, [70, 1, 300])


@pytest.mark.parametrize("P", [1, 3, 64, 100, 1024])
@pytest.mark.parametrize("order", ["rows", "heads"])
def test_attention_page_sizes(qp, P, order):
    check_q8(qp, BF16, 12, 2, 128, P, [257, 40, 1, 999], order)


@pytest.mark.parametrize("t,length", [(BF16, [40001]), (F32, [9000, 1]), (F16, [131071]), (F32, [30001, 0, 2047]), (BF16, [6000, 0, 2047])])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_long(qp, t, length, hd):
    check_q8(qp, t, 12, 2, hd, 64, length, "heads")


def test_attention_many_ragged_requests(qp):
    rng = random.Random(3)
    check_q8(qp, BF16, 14, 2, 64, 16, [rng.choice([0, 1, 5, rng.randint(1, 400)]) for _ in range(700)])


@pytest.mark.parametrize("t", [F32, BF16, F16])
def test_attention_values_of_every_size(qp, t):
    """Scales from f16's subnormal numbers to its largest ones; a request whose V stands on weights beside a dominant key."""
    def change(q, parts, table):
        parts[3].copy_(torch.logspace(-7, 4.5, parts[3].numel(), device="cuda").view_as(parts[3]).half())
        parts[2][0] = 2.0 ** -24
    check_q8(qp, t, 14, 2, 64, 16, [100, 300], change=change)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-4, 1e4])
@pytest.mark.parametrize("t", [F32, BF16])
def test_attention_queries_of_every_size(qp, t, size):
    def change(q, parts, table):
        q.mul_(size)
        parts[2].copy_(parts[2] / max(size, 0.01))
    check_q8(qp, t, 12, 2, 128, 16, [100, 30], change=change)


@pytest.mark.parametrize("t", [F32, BF16])
def test_attention_rising_scores(qp, t):
    """Keys that grow along the request: the maximum moves unit after unit."""
    def change(q, parts, table):
        q.fill_(1)
        for r, row in enumerate(table.tolist()):
            for i, page in enumerate(row):
                if 0 <= page < parts[0].shape[0]:
                    parts[0][page] = min(127, 4 + i)
                    parts[2][page] = 0.01
    check_q8(qp, t, 14, 2, 64, 16, [1500, 100], change=change)


def test_attention_scale_and_strides(qp):
    check_q8(qp, BF16, 14, 2, 64, 16, [100, 30], scale=0.03)
    nh, nkv, hd, P, length = 14, 2, 64, 16, [90, 33]
    q, parts, table = q8_case(1, BF16, nh, nkv, hd, P, length)
    want = qp.op_paged_attention_q8(q, qp.PagedCacheQ8(*parts), table, dev(length), nh)
    wide = torch.zeros(2, nh * hd + 24, dtype=BF16, device="cuda")
    wide[:, :nh * hd] = q
    big = torch.full((2, table.shape[1] + 5), -1, dtype=I32, device="cuda")
    big[:, :table.shape[1]] = table
    # codes and scales of a larger pool, rows and heads apart
    def spread(x, more):
        n, p, h, d = x.shape
        y = torch.zeros(n + 1, p + 1, h + 1, more, dtype=x.dtype, device="cuda")[1:, 1:, 1:, :d]
        return y.copy_(x)
    k, v = (spread(x, hd + 16) for x in parts[:2])
    ks, vs = (spread(x, 8) for x in parts[2:])
    out = torch.full((2, nh * hd + 8), 5.0, dtype=BF16, device="cuda")
    got = qp.op_paged_attention_q8(wide[:, :nh * hd], qp.PagedCacheQ8(k, v, ks, vs), big[:, :table.shape[1]], dev(length), nh, out=out[:, :nh * hd])
    assert torch.equal(got, want) and (out[:, nh * hd:] == 5).all()


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_attention_refuses_requests_on_the_device(qp, t):
    nh, nkv, hd, P = 14, 2, 64, 16
    length = [40, 300, 64, 20]
    q, parts, table = q8_case(1, t, nh, nkv, hd, P, length)
    cache = qp.PagedCacheQ8(*parts)
    want = qp.op_paged_attention_q8(q, cache, table, dev(length), nh)
    work = qp.op_paged_attention_q8_workspace(cache, 4, nh)
    for what in ("negative", "long", "page", "negative page", "last page"):
        ln, tb = list(length), table.clone()
        if what == "negative":
            ln[1] = -1
        elif what == "long":
            ln[1] = table.shape[1] * P + 1
        else:
            tb[1, 18 if what == "last page" else 3] = -1 if what == "negative page" else parts[0].shape[0]
        out, lse, status = torch.full_like(q, 5), torch.full((4, nh), 5.0, device="cuda"), status_word()
        qp.op_paged_attention_q8(q, cache, tb, dev(ln), nh, out=out, lse=lse, workspace=work, status=status)
        assert int(status) == -2
        assert (out[1] == 5).all() and (lse[1] == 5).all()
        keep = [0, 2, 3]
        close(out[keep], want[keep], 4 * half(t) * want[keep].double().abs() + 1e-6)
        # the workspace is as good as new
        assert torch.equal(qp.op_paged_attention_q8(q, cache, table, dev(length), nh, workspace=work), want)


def test_offsets_past_32_bits(qp):
    """A pool of more than 4 GiB of codes: the last pages are stored to, read and attended to."""
    nh, nkv, hd, P = 8, 4, 128, 256
    n_pages = 2 ** 32 // (P * nkv * hd) + 3
    k, v = (torch.zeros(n_pages, P, nkv, hd, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages, P, nkv, hd // 32, dtype=F16, device="cuda") for _ in range(2))
    cache = qp.PagedCacheQ8(k, v, ks, vs)
    n = 100
    g = gen(8)
    qkv = torch.randn(n, (nh + 2 * nkv) * hd, generator=g, device="cuda")
    slot = (n_pages - 1) * P + torch.arange(n, device="cuda", dtype=I32)
    q = qp.op_rope_paged_store_q8(qkv, qp.RopeTable(hd), dev(list(range(n))), slot, cache, nh)
    kk, vv = qp.op_paged_read_q8(cache, slot)
    assert torch.equal(vv, values(*(x.to("cuda") for x in codec(qkv[:, (nh + nkv) * hd:].view(n, nkv, hd)))).view(n, -1))
    got = qp.op_paged_attention_q8(q[-1:], cache, dev([[n_pages - 1]]), dev([n]), nh)
    table = dev([[0]])
    want = attention_by_definition(q[-1:], *(x.view(1, n, nkv, hd) for x in (kk, vv)), table, [n], nh, 1 / math.sqrt(hd))
    close(got.view(1, nh, hd), want[0], q8_tolerance(F32, hd, [n], want)[0])


def test_streams_and_captured_graphs(qp):
    """Two graphs captured on one side stream with a workspace each, replayed with other inputs, and calls at once on two
    streams: each has what a plain call gives."""
    nh, nkv, hd, P = 14, 2, 64, 16
    length = [300, 1, 0, 777]
    q, parts, table = q8_case(4, BF16, nh, nkv, hd, P, length)
    cache, ln = qp.PagedCacheQ8(*parts), dev(length)
    slots = dev([1, 2, -1, 40])
    side = torch.cuda.Stream()
    graphs = []

    def both():
        return (qp.op_paged_attention_q8(q, cache, table, ln, nh), *qp.op_paged_read_q8(cache, slots, dtype=BF16))

    for i in range(2):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = both()
        graphs.append((graph, got))
    q.copy_(torch.randn(4, nh * hd, device="cuda"))
    ln.copy_(dev([299, 0, 0, 500]))
    slots.copy_(dev([3, -1, 4, 5]))
    torch.cuda.synchronize()
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = both()
    for _, got in graphs:
        assert all(torch.equal(a.nan_to_num(7), b.nan_to_num(7)) for a, b in zip(got, want))
    other = torch.cuda.Stream()
    for s in (side, other):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(20):
        for s in (side, other):
            with torch.cuda.stream(s):
                got.append(both())
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a.nan_to_num(7), b.nan_to_num(7)) for a, b in zip(one, want))


def test_shared_pages_and_repeats(qp):
    """Requests that share pages, and the same call again: bit for bit."""
    nh, nkv, hd, P = 28, 4, 128, 16
    q, parts, table = q8_case(6, F16, nh, nkv, hd, P, [2000, 2000, 7])
    table[1] = table[0]
    q[1] = q[0]
    cache = qp.PagedCacheQ8(*parts)
    first = qp.op_paged_attention_q8(q, cache, table, dev([2000, 2000, 7]), nh)
    for _ in range(5):
        assert torch.equal(qp.op_paged_attention_q8(q, cache, table, dev([2000, 2000, 7]), nh), first)
    close(first[1], first[0], 2 * half(F16) * first[0].double().abs() + 1e-6)


def test_a_workspace_serves_other_sizes_and_types(qp):
    nh, nkv, hd, P = 14, 2, 64, 16
    work = None
    for i in range(2):
        for t, length in ((BF16, [3000]), (F32, [5] * 90), (F16, [700, 0, 64, 129]), (F32, [20000])):
            q, parts, table = q8_case(i, t, nh, nkv, hd, P, length)
            cache = qp.PagedCacheQ8(*parts)
            work = work or qp.op_paged_attention_q8_workspace(cache, 1, nh)
            got = qp.op_paged_attention_q8(q, cache, table, dev(length), nh, workspace=work)
            assert torch.equal(got, qp.op_paged_attention_q8(q, cache, table, dev(length), nh))
    with pytest.raises(qp.MinferError, match="got one of op_paged_attention_q8"):
        plain = torch.zeros(4, 16, 2, 64, device="cuda")
        qp.op_paged_attention(torch.zeros(1, 896, device="cuda"), qp.PagedCache(plain, plain.clone()), dev([[0]]), dev([1]), 14, workspace=work)


@pytest.mark.parametrize("captured", [False, True])
def test_a_batch_served_step_by_step(qp, captured):
    """Page tables, RoPE with the quantizing store, attention and rows read back, step by step: attention is that of the rows
    read back, and those are the ones that were stored, whatever pages they moved through."""
    nh, nkv, hd, P, n, W = 4, 2, 64, 16, 5, 8
    width, max_tokens, n_pages = (nh + 2 * nkv) * hd, 160, 24
    rng = random.Random(12)
    g = gen(12)
    parts = pool(g, n_pages, P, nkv, hd)
    for x in parts[2:]:
        x.fill_(math.nan)
    cache, rope = qp.PagedCacheQ8(*parts), qp.RopeTable(hd, 32, 1e4, "interleaved", "linear", 2.0)
    ln, target = torch.zeros(n, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda")
    table = torch.full((n, W), -1, dtype=I32, device="cuda")
    free, n_free = torch.arange(n_pages, dtype=I32, device="cuda"), dev([n_pages])
    qkv, status = torch.zeros(max_tokens, width, device="cuda"), status_word()
    every = torch.arange(n_pages * P, dtype=I32, device="cuda")
    s_start, s_pos, s_slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (n + 1, max_tokens, max_tokens))
    s_q = torch.zeros(max_tokens, nh * hd, device="cuda")

    def step():
        start, pos, slot, _ = qp.op_page_tables(ln, target, P, table, free, n_free, n_pages, max_tokens, out=(s_start, s_pos, s_slot, n_free), status=status)
        q = qp.op_rope_paged_store_q8(qkv, rope, pos, slot, cache, nh, out=s_q, status=status)
        last = q[(start[1:].long() - 1).clamp(min=0)]
        o = qp.op_paged_attention_q8(last, cache, table, target, nh, status=status)
        ln.copy_(target)
        return last, o, *qp.op_paged_read_q8(cache, every, status=status)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = step()
    f, scale = rope_frequencies(32, 1e4, "linear", 2.0, 0)
    held = [torch.zeros(0, 2, nkv, hd, device="cuda") for _ in range(n)]  # the rows as they were read back when they were new
    have = [0] * n
    for i in range(12):
        want = []
        for r in range(n):
            kind = rng.choice(["prompt", "one", "one", "one", "back", "over"])
            want.append(min(64, {"prompt": have[r] + rng.randint(1, 30), "one": have[r] + 1, "back": max(0, have[r] - rng.randint(0, 20)), "over": 0}[kind]))
        new = [max(0, b - a) for a, b in zip(have, want)]
        qkv.fill_(math.nan)
        qkv[:sum(new)] = torch.randn(sum(new), width, generator=g, device="cuda")
        target.copy_(dev(want))
        if captured:
            graph.replay()
        else:
            result = step()
        last, o, k, v = result
        assert int(status) == 0
        at = 0
        for r in range(n):
            rows = [int(table[r, p // P]) * P + p % P for p in range(want[r])]
            got = torch.stack([x[rows].view(-1, nkv, hd) for x in (k, v)], 1)
            y, _ = rope_by_formula(qkv[at:at + new[r]], nh, nkv, hd, torch.arange(have[r], have[r] + new[r], device="cuda"), f, scale, "interleaved")
            at += new[r]
            kept = min(have[r], want[r])
            assert torch.equal(got[:kept], held[r][:kept])
            fresh = torch.stack([y[:, nh:nh + nkv], y[:, nh + nkv:]], 1)
            if len(fresh):
                top = fresh.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, -1, 32).flatten(-2)
                close(got[kept:], fresh, top * (0.5 / 127 + 2.0 ** -11 + 2.0 ** -18))
            held[r] = got
            if want[r]:
                s = torch.einsum("hgd,jhd->hgj", last[r].double().view(nkv, nh // nkv, hd), got[:, 0].double()) / math.sqrt(hd)
                exact = torch.einsum("hgj,jhd->hgd", torch.softmax(s, -1), got[:, 1].double()).flatten()
                size = float(last[r].double().abs().sum() / math.sqrt(hd)) * 6
                close(o[r], exact, 6 * (2 * size * 2.0 ** -20 + 2.0 ** -18))
            else:
                assert (o[r] == 0).all()
        have = want


def test_a_quantized_context_is_extended_by_the_prompt_attention(qp):
    """Rows read back as f32 regions serve op_attention, the prompt's: the next chunk of a request whose first rows are in the
    quantized cache."""
    nh, nkv, hd, P, n, more = 14, 2, 64, 16, 100, 30
    g = gen(21)
    parts = pool(g, 10, P, nkv, hd, amp=0.02)
    cache = qp.PagedCacheQ8(*parts)
    slot = torch.randperm(160, generator=g, device="cuda")[:n].to(I32)
    K, V = (torch.zeros(n + more, nkv * hd, device="cuda") for _ in range(2))
    qp.op_paged_read_q8(cache, slot, out=(K[:n], V[:n]))
    K[n:], V[n:] = torch.randn(more, nkv * hd, generator=g, device="cuda"), torch.randn(more, nkv * hd, generator=g, device="cuda")
    q = torch.randn(more, nh * hd, generator=g, device="cuda")
    pos = dev(list(range(n, n + more)))
    got = qp.op_attention(q, pos, K, V, nh, nkv, hd)
    kk, vv = (x.double().view(-1, nkv, hd) for x in (K, V))
    s = torch.einsum("thgd,jhd->thgj", q.double().view(more, nkv, nh // nkv, hd), kk) / math.sqrt(hd)
    s.masked_fill_(torch.arange(n + more, device="cuda") > pos[:, None, None, None], -math.inf)
    want = torch.einsum("thgj,jhd->thgd", torch.softmax(s, -1), vv).reshape(more, nh * hd)
    close(got, want, 2e-5 * float(want.abs().max()))


def test_the_readmes_quantized_step(qp):
    """The README's step over a quantized cache: requests of a prompt, of one token and of none, down to their tokens."""
    nh, nkv, hd, P, V, n_pages = 4, 2, 64, 16, 300, 12
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    block = next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "op_paged_attention_q8" in b)
    g = gen(21)
    codes, scales = torch.zeros(2, n_pages, P, nkv, hd, dtype=torch.int8, device="cuda"), torch.zeros(2, n_pages, P, nkv, 2, dtype=F16, device="cuda")
    table, free, n_free = torch.full((3, 4), -1, dtype=I32, device="cuda"), torch.arange(n_pages, dtype=I32, device="cuda"), dev([n_pages])
    logits = torch.randn(3, V, generator=g, device="cuda")
    s = dict(qp=qp, rope=qp.RopeTable(hd), n_head=nh, bias=None, table=table, logits=logits, k_codes=codes[0], v_codes=codes[1], k_scales=scales[0],
             v_scales=scales[1], temperature=torch.tensor([0.0, 1.0, 0.5], device="cuda"), top_k=dev([0, 1, 0]), top_p=torch.tensor([1.0, 1.0, 0.9], device="cuda"),
             min_p=torch.zeros(3, device="cuda"), u=torch.tensor([0.5, 0.9, -1.0], device="cuda"))
    have = [0, 0, 0]
    for want in ([30, 7, 0], [31, 8, 0], [32, 8, 0]):
        status = status_word()
        start, pos, slot, n_free = qp.op_page_tables(dev(have), dev(want), P, table, free, n_free, n_pages, 40, status=status)
        slots = [[int(table[r, p // P]) * P + p % P for p in range(want[r])] for r in range(3)]
        s.update(start=start, pos=pos, slot=slot, rows=dev(want), status=status, slots=dev(slots[0] + slots[1]),
                 qkv=torch.randn(40, (nh + 2 * nkv) * hd, generator=g, device="cuda"))
        exec(block, s)
        k, v = (x.double().view(-1, nkv, hd).split(want[:2]) for x in (s["k"], s["v"]))
        last = s["q"][(start[1:].long() - 1).clamp(min=0)].double().view(3, nkv, nh // nkv, hd)
        for r in range(2):
            assert (k[r] != 0).any() and (v[r] != 0).any()
            p = torch.softmax(torch.einsum("hgd,jhd->hgj", last[r], k[r]) / math.sqrt(hd), -1)
            # (as in the test above: |q|, |k|, |v| < 6, a score's error 2^-20 of its sum of sizes)
            size = float(last[r].abs().sum() / math.sqrt(hd)) * 6
            close(s["o"][r], torch.einsum("hgj,jhd->hgd", p, v[r]).flatten(), 6 * (2 * size * 2.0 ** -20 + 2.0 ** -18))
        assert (s["o"][2] == 0).all()
        assert s["token"].tolist() == [int(logits[0].argmax()), int(logits[1].argmax()), -1] and (s["logprob"] == 0).all()
        have = want


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_small_values_beside_large_queries(qp, t, hd):
    """A query is held to steps of 2^-38 of its head's largest value (a power of two here, the worst case), so to 2^-39 of it: values
    half way between two steps under keys that do not look at the largest one.  All steps are rounded the same way."""
    nh, P = 4, 16
    codes, scales = torch.zeros(1, P, nh, hd, dtype=torch.int8, device="cuda"), torch.ones(1, P, nh, hd // 32, dtype=F16, device="cuda")
    codes[0, 0, :, 1:] = 127
    q = torch.empty(1, nh, hd, device="cuda")
    q[:] = (2 * (torch.arange(hd, device="cuda") % 31) + 0.5) * 2.0 ** -38
    q[..., 0] = 1
    scale = 2.0 ** 20
    lse = torch.empty(1, nh, device="cuda")
    qp.op_paged_attention_q8(q.view(1, -1).to(t), qp.PagedCacheQ8(codes, codes.clone(), scales, scales.clone()), dev([[0]]), dev([1]), nh, scale=scale, lse=lse)
    want = (q[..., 1:].to(t).double() * 127).sum(-1) * scale
    lost = (hd - 1) * 127 * scale * 2.0 ** -39
    assert float(lost) > 2.0 ** -8  # (far more than the sums' own roundings)
    close(lse, want, lost + want.abs() * ((hd // 8 + 2) * 2.0 ** -23 + 4 * U) + 8 * U)


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_small_scales_beside_large_ones(qp, t, hd):
    """A weight times its row's scale is held to steps of 2^-38 of the request's largest scale so far, at worst: rows of subnormal scales half way
    between two steps, all rounded the same way, beside one of a large scale that weighs next to nothing."""
    nh, P, n = 4, 16, 9
    k, v = (torch.zeros(1, P, nh, hd, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(1, P, nh, hd // 32, dtype=F16, device="cuda") for _ in range(2))
    k[0, 0] = -100  # the first row scores -100, the others 0
    v[0, :n] = 127
    large = 2.0 ** 15 + 2.0 ** 5  # just past a power of two
    small = (4 * torch.arange(1, n, device="cuda") + 1) * 2.0 ** -24
    vs[0, 0], vs[0, 1:n] = large, small[:, None, None].to(F16)
    q = torch.zeros(1, nh, hd, device="cuda")
    q[..., 0] = 1
    o = qp.op_paged_attention_q8(q.view(1, -1).to(t), qp.PagedCacheQ8(k, v, ks, vs), dev([[0]]), dev([n]), nh, scale=1.0)
    p = torch.exp(torch.tensor([-100.0] + [0.0] * (n - 1), dtype=torch.float64, device="cuda"))
    want = (127 * (p * torch.cat([torch.tensor([large], device="cuda"), small]).double()).sum() / p.sum()).expand(1, nh * hd)
    lost = 127 * 2.0 ** -39 * large
    assert lost > 2.0 ** -8 * float(want.abs().max())  # (far more than the sums' own roundings)
    close(o, want, lost + want.abs() * (2.0 ** -20 + (0 if t == F32 else half(t))) + (2.0 ** -25 if t == F16 else 0))
