"""The batch operators on the GPU at their edges: values, sizes, layouts and
refusals that the plain cases do not reach, against 64-bit definitions."""
import math
import os
import re

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_batch import (BF16, F16, F32, I32, ROPE_CASES, U, attention_by_definition, attention_case, check_logprobs,  # noqa: E402, F401
                            close, dev, gen, half, qp, run_tables, status_word, tables_by_hand, tables_case)
from test_gpu_batch import test_rope_paged_store as rope_against_the_formula  # noqa: E402


# ------------------------------------------------------------------ paged attention: the weights' bits
def weight_tolerance(t, want, m, units):
    """As attention_tolerance for the scores and sums, with what two 16-bit
    numbers hold of a weight.  The upper one is at most p and leaves at most
    2^-7 p (bf16, truncated) or 1.25 * 2^-10 p (f16); the lower one is rounded,
    by half a step: 2^-15 p, or 1.25 * 2^-21 p and a step of f16's smallest numbers
    under weights raised by 2^15, 2^-39.  A warp adds its `units` units with two MMAs each, whose sums of 17 terms are
    truncated to 24 bits or more.  f32: the halves' 20 U, in scores and weights."""
    o, lse, mean, size, top = want
    hd = o.shape[-1]
    m = torch.tensor(m, dtype=torch.float64, device="cuda").view(-1, 1, 1)  # keys of each request
    split = 20 * U if t == F32 else 0
    score = size * ((hd // 8 + 2) * 2.0 ** -23 + split + 4 * U) + 8 * U
    weight = {BF16: 2.0 ** -15, F16: 1.25 * 2.0 ** -21, F32: 20 * U}[t]
    rel = 2 * score + weight + (32 + 6 * torch.log2(m.clamp(min=2))) * U + 2 * units * 17 * 2.0 ** -23
    return half(t) * o.abs() + rel * mean + (m * 2.0 ** -39 * top + 2.0 ** -25 if t == F16 else 0)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("m", [2, 33, 600])
def test_paged_attention_weights_between_two_16_bit_numbers(qp, t, m):
    """Every other key's weight lies between two neighbours of the cache's type,
    and values of opposite sign leave little but what its rounding moves."""
    nh, nkv, hd, P = 4, 2, 64, 16
    q, k, v, table = attention_case(1, t, nh, nkv, hd, P, [m], poison=False)
    q.zero_(), k.zero_()
    q[:, ::hd] = 1.0
    pages = table[0].long()
    kk, vv = (torch.zeros(len(pages) * P, nkv, hd, device="cuda") for _ in range(2))
    kk[1::2, :, 0] = -1.0
    vv[0::2], vv[1::2] = 1.0, -1.0
    k[pages], v[pages] = (x.view(-1, P, nkv, hd).to(t) for x in (kk, vv))
    for scale in (2.0 ** -9, 2.0 ** -12, 0.7, 1.9):
        o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh, scale=scale)
        want = attention_by_definition(q, k, v, table, [m], nh, scale)
        close(o.view(1, nh, hd), want[0], weight_tolerance(t, want, m, 2))


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("m", [70, 2000])
@pytest.mark.parametrize("gap", [9.0, 14.0, 18.0, 21.0])
@pytest.mark.parametrize("sink", [0, 40])
def test_paged_attention_tail_beside_a_dominant_key(qp, t, m, gap, sink):
    """One key holds nearly all of the weight and a value of zero: the result is the sum of the others' small weights."""
    nh, nkv, hd, P = 14, 2, 64, 16
    q, k, v, table = attention_case(2, t, nh, nkv, hd, P, [m], poison=False)
    q.zero_()
    q[:, ::hd] = 1.0
    pages = table[0].long()
    kk, vv = (x[pages].reshape(-1, nkv, hd).float() for x in (k, v))
    kk[:, :, 0] = torch.rand(kk.shape[0], nkv, generator=gen(m), device="cuda")
    kk[sink, :, 0] = gap + 1
    vv = 1000 + 100 * vv
    vv[sink] = 0
    k[pages], v[pages] = (x.view(-1, P, nkv, hd).to(t) for x in (kk, vv))
    lse = torch.empty(1, nh, device="cuda")
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh, scale=1.0, lse=lse)
    want = attention_by_definition(q, k, v, table, [m], nh, 1.0)
    close(o.view(1, nh, hd), want[0], weight_tolerance(t, want, m, 2))
    # an infinity under a weight of either size is one
    k2, v2 = k.clone(), v.clone()
    v2[int(pages[1]), 3, :, 5], v2[int(pages[sink // P]), sink % P, :, 6] = math.inf, -math.inf
    o2 = qp.op_paged_attention(q, qp.PagedCache(k2, v2), table, dev([m]), nh, scale=1.0).view(nh, hd)
    assert (o2[:, 5] == math.inf).all() and (o2[:, 6] == -math.inf).all()
    keep = [d for d in range(hd) if d not in (5, 6)]
    assert torch.equal(o2[:, keep], o.view(nh, hd)[:, keep])


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_paged_attention_weights_of_zero(qp, t):
    """Keys a thousand below the largest score weigh nothing, however large their values."""
    nh, nkv, hd, P, m = 4, 2, 64, 16, 50
    q, k, v, table = attention_case(4, t, nh, nkv, hd, P, [m], poison=False)
    q.zero_(), k.zero_()
    q[:, ::hd] = 1.0
    v[:] = torch.finfo(t).max / 2
    k[int(table[0, 1]), 2, :, 0] = 1000
    v[int(table[0, 1]), 2] = 0.25
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh, scale=1.0)
    assert (o == 0.25).all()


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("m", [1, 50, 5000])
def test_paged_attention_tiny_values(qp, t, m):
    """Values around 2^-100: the sums of a request's weights times them keep their bits."""
    nh, nkv, hd, P = 4, 2, 64, 16
    q, k, v, table = attention_case(4, t, nh, nkv, hd, P, [m], poison=False)
    v *= 2.0 ** -100
    q *= 0.5
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh)
    want = attention_by_definition(q, k, v, table, [m], nh, 1 / 8)
    close(o.view(1, nh, hd), want[0], weight_tolerance(t, want, m, 2))


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_paged_attention_largest_values(qp, t, sign):
    """Values, and keys and queries, at and next to the largest finite one of the type, weights from 1 to small ones."""
    nh, nkv, hd, P, m = 4, 2, 64, 16, 90
    top = torch.finfo(t).max
    q, k, v, table = attention_case(4, t, nh, nkv, hd, P, [m])
    v[table[0].long()] = sign * top
    v[int(table[0, 2]), 5] = sign * top * (1 - torch.finfo(t).eps)
    v[int(table[0, -1]), m % P:] = math.nan
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh).view(nh, hd)
    # a mean of equal numbers: their roundings, and the last one may reach the type's infinity
    assert ((o.double() * sign >= top * (1 - 2.0 ** -7)) & ((o * sign).float() > 0)).all() and not o.isnan().any()
    # one key of the largest size in a dim where the query is tiny: scores stay ordinary
    q, k, v, table = attention_case(5, t, nh, nkv, hd, P, [m])
    q[:, ::hd] = float(torch.finfo(t).tiny)
    k[int(table[0, 1]), 7, :, 0] = sign * top
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh)
    want = attention_by_definition(q, k, v, table, [m], nh, 1 / 8)
    close(o.view(1, nh, hd), want[0], weight_tolerance(t, want, m, 2))
    # the same size in the query
    q, k, v, table = attention_case(6, t, nh, nkv, hd, P, [m], poison=False)
    k[..., 0] = 0
    k[int(table[0, 1]), 7, :, 0] = float(torch.finfo(t).tiny)
    q[:, ::hd] = sign * top
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh)
    want = attention_by_definition(q, k, v, table, [m], nh, 1 / 8)
    close(o.view(1, nh, hd), want[0], weight_tolerance(t, want, m, 2))


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_paged_attention_infinite_keys_and_values(qp, t):
    """A score of -inf weighs nothing: the result is that without the key.  A value of +-inf that weighs something makes
    its dim infinite, and nothing else.  A request of which every score is -inf has zeros and an lse of -inf."""
    nh, nkv, hd, P, m = 4, 2, 64, 16, 100
    q, k, v, table = attention_case(6, t, nh, nkv, hd, P, [m, m], poison=False)
    q[:, ::hd] = 1.0
    drop = [0, 17, 18, 60, 99]
    keep = [j for j in range(m) if j not in drop]
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    n = -(-len(keep) // P)
    for x, x2 in ((k, k2), (v, v2)):
        rows = x[table[0].long()].reshape(-1, nkv, hd)[keep]
        x2[table[0, :n].long()] = torch.cat([rows, rows.new_zeros(n * P - len(keep), nkv, hd)]).view(n, P, nkv, hd)
    want = attention_by_definition(q[:1], k2, v2, table[:1, :n], [len(keep)], nh, 1 / 8)
    for j in drop:
        k[int(table[0, j // P]), j % P, :, 0] = -math.inf
    lse = torch.empty(2, nh, device="cuda")
    cache = qp.PagedCache(k, v)
    o = qp.op_paged_attention(q, cache, table, dev([m, m]), nh, lse=lse)
    close(o[:1].view(1, nh, hd), want[0], weight_tolerance(t, want, m, 2))
    v[int(table[0, 3]), 4, :, 5], v[int(table[0, 2]), 4, :, 9] = math.inf, -math.inf
    o2 = qp.op_paged_attention(q, cache, table, dev([m, m]), nh).view(2, nh, hd)
    assert (o2[0, :, 5] == math.inf).all() and (o2[0, :, 9] == -math.inf).all()
    o2[0, :, [5, 9]] = o.view(2, nh, hd)[0, :, [5, 9]]
    assert torch.equal(o2.view(2, -1), o)
    k[table[0].long(), :, :, 0] = -math.inf
    v[table[0].long()] = 1.0
    o3 = qp.op_paged_attention(q, cache, table, dev([m, m]), nh, lse=lse)
    assert (o3[0] == 0).all() and (lse[0] == -math.inf).all() and torch.equal(o3[1], o[1])


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("m", [1500, 33])
def test_paged_attention_rising_and_falling_scores(qp, t, m):
    """Scores that rise along the request by 60 in all, or fall: the first, or last, keys' weights vanish."""
    nh, nkv, hd, P = 7, 1, 64, 16
    for lo, hi in ((-30.0, 30.0), (30.0, -30.0)):
        q, k, v, table = attention_case(5, t, nh, nkv, hd, P, [m], poison=False)
        q.zero_()
        q[:, ::hd] = 1.0
        k[table[0].long(), :, 0, 0] = torch.linspace(lo, hi, table.shape[1] * P, device="cuda").view(-1, P).to(t)
        lse = torch.empty(1, nh, device="cuda")
        o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev([m]), nh, scale=1.0, lse=lse)
        want = attention_by_definition(q, k, v, table, [m], nh, 1.0)
        close(o.view(1, nh, hd), want[0], weight_tolerance(t, want, m, 2))
        close(lse, want[1], 2 * want[3][..., 0] * (10 * 2.0 ** -23 + 24 * U) + 2.0 ** -18)


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(12, 2, 128), (32, 2, 64), (20, 1, 128)])
@pytest.mark.parametrize("m", [200, 30001])
def test_paged_attention_small_weights_of_every_layout(qp, t, nh, nkv, hd, m):
    """The tail beside a dominant key in blocks of 8 and 16 heads, over one share, joins of one and of two levels."""
    P, length, rows = 16, [m, 0, 40], (0, 2)
    q, k, v, table = attention_case(m, t, nh, nkv, hd, P, length, "heads")
    q.zero_()
    q[:, ::hd] = 1.0
    for r in rows:
        pages = table[r, :-(-length[r] // P)].long()
        kk, vv = (x[pages].reshape(-1, nkv, hd).float() for x in (k, v))
        kk[:, :, 0] = torch.rand(kk.shape[0], nkv, generator=gen(m), device="cuda")
        kk[length[r] // 3, :, 0] = 16
        vv = 100 + 10 * vv  # (what lies behind the last row stays NaN)
        vv[length[r] // 3] = 0
        k[pages], v[pages] = (x.view(-1, P, nkv, hd).to(t) for x in (kk, vv))
    lse = torch.empty(3, nh, device="cuda")
    o = qp.op_paged_attention(q, qp.PagedCache(k, v), table, dev(length), nh, scale=1.0, lse=lse)
    want = attention_by_definition(q, k, v, table, length, nh, 1.0)
    tol = weight_tolerance(t, want, length, 30)
    close(o.view(3, nh, hd), want[0], tol)
    # half a step of the result is the largest part of the tolerance of 16-bit caches
    if t != F32:
        assert float((tol / want[0].abs())[list(rows)].max()) < (2.0 ** -7 if t == BF16 else 2.0 ** -9)


@pytest.mark.parametrize("m", [131071])
def test_paged_attention_long_request_with_large_results(qp, m):
    """Values around 1, so that a part of the keys left out would show: the result stands far above its tolerance."""
    nh, nkv, hd, P = 14, 2, 64, 64
    q, k, v, table = attention_case(3, F16, nh, nkv, hd, P, [m])
    q *= 0.5
    v[table[0].long()] = (1 + 0.5 * v[table[0].long()].float()).to(F16)
    v[int(table[0, -1]), m % P:] = math.nan
    cache = qp.PagedCache(k, v)
    work = qp.op_paged_attention_workspace(cache, 1, nh)
    lse = torch.empty(1, nh, device="cuda")
    o = qp.op_paged_attention(q, cache, table, dev([m]), nh, lse=lse, workspace=work)
    want = attention_by_definition(q, k, v, table, [m], nh, 1 / 8)
    tol = weight_tolerance(F16, want, m, 12)
    assert float((tol / want[0].abs()).max()) < 2.0 ** -9
    close(o.view(1, nh, hd), want[0], tol)
    # counters of shares, of groups, of the second level: all back at zero
    shares = 16 * 63
    assert int(work.buffer[:4 * (2 * shares + shares // 16 + 1)].max()) == 0
    assert torch.equal(o, qp.op_paged_attention(q, cache, table, dev([m]), nh, workspace=work))


# ------------------------------------------------------------------ refused steps
def litter(value, dtype, sizes):
    """Freed memory of these sizes that holds `value`: what a fresh tensor that nobody fills is likely to show."""
    junk = [torch.full((n,), value, dtype=dtype, device="cuda") for n in sizes for _ in range(8)]
    torch.cuda.synchronize()
    del junk


def test_a_refused_page_tables_step_returns_the_old_depth(qp):
    """Without `out`, as a loop that rebinds n_free to what it gets: a step that finds too few pages, then one that fits."""
    P, W, n_pages = 16, 4, 6
    table, free, n_free = dev([[0, -1, -1, -1], [1, 2, -1, -1]]), dev([3, 4, 5, -1, -1, -1]), dev([3])
    litter(2, I32, (1, 3, 80))
    status = status_word()
    start, pos, slot, n_free = qp.op_page_tables(dev([16, 32]), dev([64, 49]), P, table, free, n_free, n_pages, 80, status=status)
    assert int(status) == -7 and n_free.tolist() == [3]
    assert start.tolist() == [0, 0, 0] and set(pos.tolist()) == set(slot.tolist()) == {-1}
    status.zero_()
    got = qp.op_page_tables(dev([16, 32]), dev([17, 0]), P, table, free, n_free, n_pages, 80, status=status)
    want = tables_by_hand([16, 32], [17, 0], P, [[0, -1, -1, -1], [1, 2, -1, -1]], [3, 4, 5, -1, -1, -1], 3, 80)
    assert int(status) == 0
    assert (table.tolist(), free.tolist(), int(got[3]), *(x.tolist() for x in got[:3])) == want


def test_fresh_outputs_of_skipped_rows(qp):
    """Without `out`, rows that are not written are zero (token ids -1), so sums over a padded batch hold."""
    x, k = torch.randn(6, 500, device="cuda"), 4
    for t in (F32, I32):
        litter(9, t, (6, 24, 36))
    status = status_word()
    logprob, entropy, top_ids, top_logprobs = qp.op_token_logprobs(x, dev([3, -1, 500, 7, -5, 499]), k, status=status)
    assert int(status) == -3
    skipped, live = [1, 2, 4], [0, 3, 5]
    assert (logprob[skipped] == 0).all() and (entropy[skipped] == 0).all()
    assert (top_ids[skipped] == -1).all() and (top_logprobs[skipped] == 0).all()
    for got, want in zip((logprob, entropy, top_ids, top_logprobs), qp.op_token_logprobs(x[live], dev([3, 7, 499]), k)):
        assert torch.equal(got[live], want)
    none, entropy0, top_ids0, top_logprobs0 = qp.op_token_logprobs(x, None, k)
    assert none is None and torch.equal(top_ids0[live], top_ids[live]) and torch.equal(top_logprobs0[live], top_logprobs[live])
    assert torch.equal(entropy0[live], entropy[live]) and qp.op_token_logprobs(x, dev([1] * 6), 0)[2].shape == (6, 0)
    nh, nkv, hd, length = 4, 2, 64, [30, 40, 0]
    for t in (F32, F16, BF16):
        q, kk, v, table = attention_case(7, t, nh, nkv, hd, 16, length)
        cache = qp.PagedCache(kk, v)
        table[1, 1] = -1
        litter(9, t, (3 * nh * hd,))
        status.zero_()
        o = qp.op_paged_attention(q, cache, table, dev(length), nh, status=status)
        assert int(status) == -2 and (o[1:] == 0).all() and (o[0] != 0).any()


def readme_step():
    """The README's step of a batch, from its page tables on."""
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    block = next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "op_page_tables" in b)
    return block[block.index("start, pos, slot"):]


@pytest.mark.parametrize("refused", [False, True])
def test_the_readmes_step(qp, refused):
    """A request is rolled back and its page goes to another one; then it is to grow again, and the other one too, which
    is done, or refused for want of a page.  Attention sees each request's own rows in both cases."""
    nh, nkv, hd, P, V = 4, 2, 64, 16, 300
    n_pages = 3 if refused else 6
    cache = qp.PagedCache(*(torch.full((n_pages, P, nkv, hd), math.nan, device="cuda") for _ in range(2)))
    s = dict(qp=qp, torch=torch, cache=cache, rope=qp.RopeTable(head_dim=hd, theta=1e4), page_size=P, n_pages=n_pages, n_head=nh, bias=None,
             table=torch.full((2, 4), -1, dtype=I32, device="cuda"), free=torch.arange(n_pages, dtype=I32, device="cuda"), n_free=dev([n_pages]),
             logits=torch.randn(2, V, device="cuda"), ids=dev([5, 7]), max_tokens=44)
    g = gen(1)
    have, keys = [0, 0], [[], []]  # the K and V rows of each request, by the positions and slots of its steps
    for want, ok in (([20, 12], True), ([10, 12], True), ([11, 22], True), ([27, 38], not refused)):
        s.update(length=dev(have), target=dev(want), status=status_word(), qkv=torch.randn(44, (nh + 2 * nkv) * hd, generator=g, device="cuda"))
        exec(readme_step().replace("qp.check_status(status)", ""), s)
        assert int(s["status"]) == (0 if ok else -7)
        if ok:
            at = 0
            for r in range(2):
                new = max(0, want[r] - have[r])
                slots = s["slot"][at:at + new].long()
                at += new
                # the step's rows, from the cache as the store left them
                rows = torch.stack([x[slots // P, slots % P] for x in (cache.k, cache.v)], 1)
                keys[r] = torch.cat([keys[r][:min(have[r], want[r])], rows]) if len(keys[r]) else rows
            have = want
        held = [min(a, b) for a, b in zip(have, want)]
        for r in range(2):
            k, v = keys[r][:held[r]].unbind(1)
            n = -(-held[r] // P)
            k, v = (torch.cat([x, x.new_zeros(n * P - held[r], nkv, hd)]).view(n, P, nkv, hd) for x in (k, v))
            tb = torch.arange(n, dtype=I32, device="cuda")[None]
            o = attention_by_definition(s["newest"][r:r + 1], k, v, tb, [held[r]], nh, 1 / 8)
            close(s["o"][r:r + 1].view(1, nh, hd), o[0], weight_tolerance(F32, o, held[r], 2))


def test_a_step_without_rows(qp):
    """No requests, no tokens, no logits rows: empty results of the right shapes, and outputs that are set as a step without tokens sets them."""
    nh, nkv, hd, P = 4, 2, 64, 16
    cache = qp.PagedCache(torch.zeros(3, P, nkv, hd, device="cuda"), torch.zeros(3, P, nkv, hd, device="cuda"))
    none, free, n_free = dev([]), dev([2, 1, 0]), dev([3])
    for out in (None, tuple(torch.full((m,), 9, dtype=I32, device="cuda") for m in (1, 5, 5, 1)), (dev([9]), dev([9] * 5), dev([9] * 5), n_free)):
        start, pos, slot, left = qp.op_page_tables(none, none, P, none.view(0, 4), free, n_free, 3, 5, out=out)
        assert (start.tolist(), pos.tolist(), slot.tolist(), left.tolist(), free.tolist()) == ([0], [-1] * 5, [-1] * 5, [3], [2, 1, 0])
    q = qp.op_rope_paged_store(torch.zeros(0, (nh + 2 * nkv) * hd, device="cuda"), qp.RopeTable(hd), none, none, cache, nh)
    assert q.shape == (0, nh * hd) and q.dtype == F32
    assert qp.op_paged_attention(q, cache, none.view(0, 4), none, nh, lse=torch.zeros(0, nh, device="cuda")).shape == q.shape
    logprob, entropy, top_ids, top_logprobs = qp.op_token_logprobs(torch.zeros(0, 50, device="cuda"), none, 3)
    assert logprob.shape == entropy.shape == (0,) and top_ids.shape == top_logprobs.shape == (0, 3)
    assert qp.op_token_logprobs(torch.zeros(0, 50, device="cuda"))[0] is None


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_single_rows_of_any_stride(qp, t):
    """One row out of a buffer of odd width, a cache of one KV head, of one page or of pages of one row out of odd views:
    what contiguous copies give."""
    for nh, nkv, hd, n_pages, P, m in ((4, 1, 64, 5, 16, 60), (4, 2, 64, 1, 48, 41), (6, 2, 128, 40, 1, 37)):
        g = gen(m)
        odd = lambda shape, n: torch.randn(n, generator=g, device="cuda").to(t).as_strided(  # noqa: E731
            shape, [n if d == 1 else s for d, s in zip(shape, (P * nkv * hd, nkv * hd, hd, 1))])
        n = n_pages * P * nkv * hd
        k, v = (odd((n_pages, P, nkv, hd), n + (n + 1) % 2) for _ in range(2))
        table = torch.randperm(n_pages, generator=g, device="cuda").to(I32)[None]
        qkv = torch.randn(3, (nh + 2 * nkv) * hd + 1, generator=g, device="cuda").to(t)[:1, :-1]
        out = torch.zeros(2, nh * hd + 1, dtype=t, device="cuda")[:1, :-1]
        assert all(s % 8 for s, d in zip(k.stride(), k.shape) if d == 1) and qkv.stride(0) % 8
        results = []
        for fit in (lambda x: x, lambda x: x.clone(memory_format=torch.contiguous_format)):
            kk, vv = torch.empty_strided(k.shape, k.stride(), dtype=t, device="cuda"), torch.empty_strided(v.shape, v.stride(), dtype=t, device="cuda")
            kk, vv = (kk.copy_(k), vv.copy_(v)) if fit(k) is k else (fit(k), fit(v))
            cache = qp.PagedCache(kk, vv)
            q = qp.op_rope_paged_store(fit(qkv), qp.RopeTable(hd), dev([m - 1]), dev([int(table[0, (m - 1) // P]) * P + (m - 1) % P]), cache, nh,
                                       out=fit(out))
            results.append((q.clone(), qp.op_paged_attention(q, cache, table, dev([m]), nh, out=fit(out)).clone(), kk, vv))
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert (results[0][1] != 0).any()


def test_a_workspace_belongs_to_one_operator(qp):
    """What log probabilities leave in a workspace lies where attention has counters, so the other operator's is refused."""
    nh, nkv, hd, length = 4, 2, 64, [700, 3]
    q, k, v, table = attention_case(1, BF16, nh, nkv, hd, 16, length)
    cache, x = qp.PagedCache(k, v), torch.randn(2, 5000, device="cuda")
    size = 1 << 24
    for mine in (qp.Workspace(size, "cuda"), qp.op_paged_attention_workspace(cache, 2, nh)):
        o = qp.op_paged_attention(q, cache, table, dev(length), nh, workspace=mine)
        with pytest.raises(qp.MinferError, match="one of op_token_logprobs wanted, got one of op_paged_attention"):
            qp.op_token_logprobs(x, None, 3, workspace=mine)
        assert torch.equal(o, qp.op_paged_attention(q, cache, table, dev(length), nh, workspace=mine))
    for mine in (qp.Workspace(size, "cuda"), qp.op_token_logprobs_workspace(x, 3)):
        a = qp.op_token_logprobs(x, None, 3, workspace=mine)
        with pytest.raises(qp.MinferError, match="one of op_paged_attention wanted, got one of op_token_logprobs"):
            qp.op_paged_attention(q, cache, table, dev(length), nh, workspace=mine)
        assert torch.equal(a[2], qp.op_token_logprobs(x, None, 3, workspace=mine)[2])


# ------------------------------------------------------------------ page tables: refusals in a cluster of sixteen
@pytest.mark.parametrize("what,code", [("long length", -2), ("tokens", -10), ("pages", -7), ("depth", -1), ("free id", -1), ("shared page id", -1),
                                       ("returned id", -1)])
@pytest.mark.parametrize("n", [40, 1500])
def test_page_tables_refusals_of_large_steps(qp, n, what, code):
    """Steps of more than 8,192 rows, which sixteen CTAs do: nothing changes."""
    P, W, max_tokens = 16, 24, 12000
    length, target, table, free, n_free = tables_case(n, n, P, W, ["one", "same", "back", "over"])
    for r, (a, b, row) in {3: (0, W * P, []), n - 2: (18, 19, [0, 1]), n - 1: (P * W, 3, list(range(W)))}.items():
        length[r], target[r], table[r] = a, b, row + [-7] * (W - len(row))
    free, n_free = list(range(n * W)), n * W
    if what == "long length":
        length[n - 1] = P * W + 1
    elif what == "tokens":
        length, target, table = [0] * n, [W * P] * n, [[-7] * W] * n
    elif what == "pages":
        n_free = W - 3
        length, target, table = [0] * n, [0] * (n - 1) + [W * P], [[-7] * W] * n
    elif what == "depth":
        n_free = n * W + 1
    elif what == "free id":
        free[n_free - 5] = n * W
    elif what == "shared page id":
        table[n - 2][1] = -1
    elif what == "returned id":
        table[n - 1][W - 1] = n * W
    if what == "tokens":
        max_tokens = min(max_tokens, n * W * P - 1)
    status = status_word()
    t, f, left, start, pos, slot = run_tables(qp, (length, target, table, free, n_free), P, max_tokens, False, status)
    assert int(status) == code
    assert t == table and f == free and left == -9
    assert start == [0] * (n + 1) and pos == [-1] * max_tokens and slot == [-1] * max_tokens


# ------------------------------------------------------------------ RoPE: several tokens per CTA
def rope_rows():
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
    return 2 * 2 * sms, 4 * 2 * sms  # from here on two tokens a CTA, and four


@pytest.mark.parametrize("case", range(len(ROPE_CASES)))
@pytest.mark.parametrize("which,more", [(0, -1), (0, 1), (1, 0), (1, 3)])
def test_rope_paged_store_of_many_rows(qp, case, which, more):
    """CTAs of one, two and four tokens, the last of them in part behind the rows, padding beside live rows."""
    n = rope_rows()[which] + more
    rope_against_the_formula(qp, *ROPE_CASES[case], n, "heads" if (case + more) % 2 else "rows")


@pytest.mark.parametrize("src,to", [(F32, F32), (F32, BF16), (F16, F16)])
@pytest.mark.parametrize("which", [0, 1])
def test_rope_rows_do_not_depend_on_their_neighbours(qp, src, to, which):
    """Padding, refused slots and positions in every place of a CTA: the other rows are, bit for bit, what calls of a few rows give."""
    nh, nkv, hd, P = 6, 2, 128, 16
    g = gen(which)
    n = rope_rows()[which] + 7
    width = (nh + 2 * nkv) * hd
    qkv = torch.randn(n, width, generator=g, device="cuda").to(src)
    bias, norms = torch.randn(width, generator=g, device="cuda"), [1 + torch.rand(hd, generator=g, device="cuda") for _ in range(2)]
    pages = -(-n // P)
    pos = torch.randint(0, 100000, (n,), generator=g, device="cuda").to(I32)
    slot = torch.randperm(pages * P, generator=g, device="cuda")[:n].to(I32)
    kind = torch.randint(0, 6, (n,), generator=g, device="cuda")
    kind[400:440] = 0  # whole CTAs of padding
    slot[kind == 0], pos[kind == 1], slot[kind == 2] = -1, -1, pages * P
    results, rope = [], qp.RopeTable(hd)
    for step in (n, 150):
        k, v = (torch.full((pages, P, nkv, hd), 3.0, dtype=to, device="cuda") for _ in range(2))
        out, cache = torch.full((n, nh * hd), 3.0, dtype=to, device="cuda"), qp.PagedCache(k, v)
        for i in range(0, n, step):
            status = status_word()
            qp.op_rope_paged_store(qkv[i:i + step], rope, pos[i:i + step], slot[i:i + step], cache, nh, bias=bias, q_norm=norms[0],
                                   k_norm=norms[1], out=out[i:i + step], status=status)
            assert int(status) == (-2 if ((kind[i:i + step] == 1) | (kind[i:i + step] == 2)).any() else 0)
        results.append((out, k, v))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert (results[0][0][kind < 3] == 3).all() and not (results[0][0][kind >= 3] == 3).all(1).any()


# ------------------------------------------------------------------ log probabilities: 16-bit rows, large references
HARD = ["equal", "two levels", "one left", "two left", "none left", "largest", "tiny", "peak", "zeros of both signs", "lowest", "all lowest",
        "lowest first", "masked first", "climbing"]


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("kind", HARD)
@pytest.mark.parametrize("rows,V,k", [(3, 5000, 20), (2, 151937, 32), (3, 40, 32), (650, 20001, 7)])
def test_token_logprobs_hard_rows_of_every_type(qp, t, kind, rows, V, k):
    g = gen(V)
    lowest, top = torch.finfo(t).min, torch.finfo(t).max
    x = torch.randn(rows, V, generator=g, device="cuda")
    if kind == "equal":
        x.fill_(1.25)
    elif kind == "two levels":
        x = (x > 1).float()
    elif kind == "one left":
        x.fill_(-math.inf)
        x[:, V - 1] = -3.0
    elif kind == "two left":
        x.fill_(-math.inf)
        x[:, 0], x[:, V // 2] = 2.0, 2.0
    elif kind == "none left":
        x[1].fill_(-math.inf)
    elif kind == "largest":
        x *= top / 16
    elif kind == "tiny":
        x *= torch.finfo(t).tiny * 4
    elif kind == "peak":
        x[:, 7] = 60.0
    elif kind == "zeros of both signs":
        x = torch.where(x > 0, 0.0, -0.0)
    elif kind == "lowest":
        x = torch.where(x > 1, x, lowest)
    elif kind == "all lowest":
        x.fill_(lowest)
    elif kind == "lowest first":
        x[:, :V // 3] = lowest
        x[0, :V - 3] = lowest
    elif kind == "masked first":
        x[:, :V // 3] = -math.inf
        x[0, :V - 3] = -math.inf
    elif kind == "climbing":  # through references of every size, in each row of 650 by every warp
        x += torch.linspace(-1, 1, V, device="cuda") * (50000 if t == F16 else 4e6)
    ids = (torch.arange(rows, device="cuda") * 17 % V).to(I32)
    ids[:3] = torch.tensor([0, V - 1, V // 2], device="cuda")[:rows]
    check_logprobs(qp, x.to(t), ids, k)


@pytest.mark.parametrize("t,at", [(F32, 1.0e6), (F32, 2.0 ** 20 - 8), (F32, 1.1e6), (F32, 300.0), (F32, 5e4), (F32, 1e8), (BF16, 300.0), (BF16, 1.0e6),
                                  (BF16, 1.2e6), (BF16, 3e4), (F16, 300.0), (F16, 4000.0), (F16, 32700.0), (F16, 33000.0), (F16, 65000.0)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("V", [3001, 151936])
def test_token_logprobs_around_large_references(qp, t, at, sign, V):
    """Logits a few steps around a large one: references below and above the size up to which terms are one multiply-add,
    whose rounding the sums are corrected for."""
    x = torch.randn(4, V, generator=gen(V), device="cuda")
    x = (sign * at + torch.where(torch.rand(4, V, generator=gen(1), device="cuda") < 0.5, 2 * x, 0.0)).to(t)
    x[3, 1::2] = -math.inf
    x[2, ::3] = torch.finfo(t).min
    assert torch.isfinite(x[:2]).all()
    check_logprobs(qp, x, dev([0, V - 1, V // 2, 4]), 8)


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("V", [3000, 3007, 100000])
def test_token_logprobs_nan_and_infinity_of_every_type(qp, t, V):
    x = torch.randn(6, V, generator=gen(3), device="cuda").to(t)
    x[0, 0], x[0, V - 1] = math.nan, math.inf
    x[1, 5], x[1, 9] = math.inf, math.inf
    x[2, 1:2000] = math.nan
    x[4, ::2] = -math.inf
    x[4, V - 1] = math.nan
    x[5].fill_(-math.inf)
    x[5, V // 2] = math.inf
    logprob, entropy, ids, lps = qp.op_token_logprobs(x, dev([3] * 6), 5)
    bad = [0, 1, 2, 4, 5]
    assert torch.isnan(logprob[bad]).all() and torch.isnan(entropy[bad]).all() and torch.isnan(lps[bad]).all()
    assert ids[0, :2].tolist() == [0, V - 1] and ids[1, :2].tolist() == [5, 9] and ids[2].tolist() == [1, 2, 3, 4, 5]
    assert int(ids[4, 0]) == V - 1 and ids[5].tolist() == [V // 2, 0, 1, 2, 3]
    check_logprobs(qp, x[3:4], dev([3]), 5)
