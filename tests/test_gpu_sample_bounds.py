"""What the contract of sampling promises to the last bit: how far weights may be off, draws from a random number of 0, and rows at
other addresses."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_batch import BF16, F16, F32, I32, close, gen, status_word  # noqa: E402

INF = math.inf


@pytest.fixture(scope="module")
def qp():
    import quantized_transformer_prefill_gb300 as qp
    qp.lib()
    return qp


# How far a weight may be off, as a share of itself.  With t = x log2(e) / T = whole + j / 256 + r, in units of the mantissa 2^(j/256 + r):
#   the table's entry and the sum, each the nearest multiple of 2^-30      2 x 2^-31
#   2^r as a quadratic, |r| <= 2^-9 + |t| 2^-23 (t is a sum of two f32)    0.0555 |r|^3
#   its two steps, r and the entry as f32, half a step of 2^-23 each       0.694 |r| 2^-22
#   log2(e) / T as a sum of two f32, and the rounding of t's lower part    |t| 1.5e-14
def off_by(t):
    r = 2.0 ** -9 + t * 2.0 ** -23
    return 2.0 ** -30 + 0.0555 * r ** 3 + 0.694 * r * 2.0 ** -22 + t * 1.5e-14


@pytest.mark.parametrize("far,bound", [(0.0, 2.0 ** -29), (690.0, 2.0 ** -29), (5600.0, 2.0 ** -28), (1.0e5, 2.0 ** -29)])
def test_weights_are_as_exact_as_promised(qp, far, bound):
    """Rows of two tokens with random numbers as near to the border between them as f32 has them: where that is farther away than
    the weights may be off, the draw is the definition's.  far: how many temperatures the largest logit lies from 0; from 5,678 on
    weights are taken from differences."""
    assert off_by(min(far + 43, 5721) * 1.4427 if far < 5678 else 62.1) < bound
    g = gen(int(far) + 1)
    n = 1 << 18
    rand = lambda: torch.rand(n, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    temp = torch.exp(3 * (2 * rand() - 1)).float()
    sign = torch.where(rand() < 0.5, -1.0, 1.0)
    x = torch.empty(n, 2, device="cuda")
    x[:, 0] = (far * (0.75 + 0.25 * rand()) * sign * temp.double()).float()
    x[:, 1] = (x[:, 0].double() + 12 * (2 * rand() - 1) * temp.double()).float().clamp(-far * temp, far * temp) if far else 12 * (2 * rand() - 1).float() * temp
    d = (x[:, 0].double() - x[:, 1].double()) / temp.double()
    share = 1 / (1 + torch.exp(-d))
    # two weights that are off by `bound` each move the border by 2 (1 - share) of them
    slack = share * (2 * bound * (1 - share) + 2.0 ** -43)
    u = (share + slack * 8 * (2 * rand() - 1)).float()
    u = torch.where(u < 1, u, torch.nextafter(torch.ones_like(u), torch.zeros_like(u)))
    gap = u.double() - share
    sure = gap.abs() > slack
    status = status_word()
    token, _ = qp.op_sample(x, u, temp, status=status)
    assert int(status) == 0
    want = (gap >= 0).int()
    assert torch.equal(token[sure], want[sure])
    assert int((sure & (gap.abs() < 4 * slack)).sum()) > 1000  # (some of them are near)


def first_left(x, temp=1.0, k=0, p=1.0, floor=0.0, first=False):
    """The first id of what is left of a row, and the logarithm of its share: [(id, log share)] for every length that top-p may leave when its
    border is off by 2^-30 of the whole.  A draw from a random number of 0 is one of these, and no sum of weights decides it."""
    x = x.double()
    at = torch.nonzero(x > -INF)[:, 0]
    if not len(at):
        return [(-1, -INF)]
    if temp == 0:
        return [(int(torch.nonzero(x == x.max())[0, 0]), 0.0)]
    sharp = temp if first else 1.0
    order = at[torch.sort(x[at], descending=True, stable=True).indices]
    if k > 0:
        order = order[:k]
    lengths = [len(order)]
    if p < 1:
        w = torch.exp((x[order] - x[order[0]]) / sharp)
        before, whole = w.cumsum(0) - w, w.sum()
        lengths = [max(1, int((before < (p + d) * whole).sum())) for d in (-2.0 ** -30, 2.0 ** -30)]
    got = []
    for n in range(lengths[0], lengths[-1] + 1):
        left = order[:n]
        z = x[left] - x[order[0]]
        keep = z / temp >= -60 * math.log(2)
        if floor > 0:
            keep &= torch.exp(z / sharp) >= floor
        left = left[keep].sort().values
        z = (x[left] - x[order[0]]) / temp
        got.append((int(left[0]), float(z[0] - torch.logsumexp(z, 0))))
    return got


@pytest.mark.parametrize("t,rows,V,extra", [(F32, 11, 40, 0), (BF16, 11, 5000, 3), (F16, 11, 32001, 5), (F32, 7, 151936, 0),
                                            (F32, 52, 151936, 0), (BF16, 130, 150001, 3), (F16, 400, 40000, 1)])  # the last three are streamed
@pytest.mark.parametrize("kind", ["plain", "k", "k and p", "p", "min", "large k", "hot", "all", "each its own"])
def test_a_random_number_of_0_draws_the_first_token_left(qp, t, rows, V, extra, kind):
    """However little it weighs: without a filter the first token of a row is one of 2^-20 and less of the whole, which no comparison of
    sums within their accuracy would tell from the next one."""
    from test_gpu_sample import SETTINGS, logits
    x = logits(gen(V + rows + len(kind)), rows, V, t, extra, masked=V % 2 == 1)
    x[rows // 2] = -INF
    settings = {name: [f(r) for r in range(rows)] for name, f in SETTINGS[kind].items()}
    tensor = lambda name, dt=F32: torch.tensor(settings[name], dtype=dt, device="cuda") if name in settings else None  # noqa: E731
    args = tensor("temp"), tensor("k", I32), tensor("p"), tensor("floor")
    for first in (False, True):
        status = status_word()
        token, logprob = qp.op_sample(x, torch.zeros(rows, device="cuda"), *args, temperature_first=first, status=status)
        assert int(status) == 0
        for r in range(rows):
            row = {name: a[r].item() for name, a in zip(("temp", "k", "p", "floor"), args) if a is not None}
            row["k"] = max(row.get("k", 0), 0)
            want = first_left(x[r], first=first, **row)
            assert int(token[r]) in [i for i, _ in want], (r, int(token[r]), want[:3])
            if len(want) == 1:
                close(logprob[r:r + 1], torch.tensor([want[0][1]], dtype=torch.float64, device="cuda"), 2.0 ** -28 + 2.0 ** -23 * min(abs(want[0][1]), 1e30))


@pytest.mark.parametrize("t,rows,V", [(F32, 60, 151936), (BF16, 130, 150001), (F16, 400, 40000)])
def test_streamed_rows_at_other_addresses(qp, t, rows, V):
    """Blocks of a streamed row begin where its address modulo 16 says, and a block's sum is rounded once: the same logits elsewhere may be
    drawn from differently, but only where the border lies within these roundings; at the same address modulo 16 they never are."""
    from test_gpu_sample import check, logits
    E, width = 16 // t.itemsize, V + 16
    one = logits(gen(V), rows, V, t, masked=True)
    u = torch.rand(rows, generator=gen(2), device="cuda").tolist()
    for offset in {1, E // 2, E - 1}:
        x = torch.empty(rows, width, dtype=t, device="cuda")[:, offset:offset + V]
        x.copy_(one)
        assert qp.op_sample_workspace(x) is not None
        for settings in (dict(temp=[0.9] * rows), dict(temp=[1.1] * rows, p=[0.97] * rows), dict(k=[50] * rows, p=[0.9] * rows)):
            check(qp, x, u, **settings)
    # Two tokens of 0.3 units next to a block's end, and behind them two that weigh half of the row each: with u = 0.5 the first of these is
    # drawn if the small ones count for a unit, the second if they do not.  Both are within 2^-(62 - log2 V) of the border.
    unit = 62 - math.ceil(math.log2(V))
    x = torch.empty(rows, width | 1, dtype=t, device="cuda").fill_(-INF)[:, 1:1 + V]  # every row at another address
    end, a, b = 128 * E, 640 * E + 7, V - 1
    x[:, end - 1] = x[:, end - E] = (math.log(0.3) - unit * math.log(2))
    x[:, a] = x[:, b] = 0
    half = torch.full((rows,), 0.5, device="cuda")
    assert qp.op_sample_workspace(x) is not None
    token, logprob = qp.op_sample(x, half)
    assert all(i in (a, b) for i in token.tolist())
    close(logprob, torch.full((rows,), -math.log(2), dtype=torch.float64, device="cuda"), 2.0 ** -23)
    by_address = {}
    for r in range(rows):
        by_address.setdefault(x[r].data_ptr() % 16, set()).add(int(token[r]))
    assert len(by_address) == E and all(len(tokens) == 1 for tokens in by_address.values())
    again = qp.op_sample(x, half)
    assert torch.equal(again[0], token) and torch.equal(again[1], logprob)


@pytest.mark.parametrize("rows,V", [(12, 40), (12, 5000), (6, 151936), (60, 151936)])
def test_negative_zeros_are_zeros(qp, rows, V):
    """As random numbers (they mark no padding), temperatures, top_p and min_p."""
    from test_gpu_sample import logits
    x = logits(gen(V + rows), rows, V, F32, 1)
    u = torch.rand(rows, generator=gen(1), device="cuda")
    zero, one = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    k = torch.tensor([[0, 50, 1000][r % 3] for r in range(rows)], dtype=I32, device="cuda")
    for first in (False, True):
        for args in ((zero, one, None, None, None), (zero, one, k, 0.9 * one, None), (u, one, k, zero, None), (u, one, None, zero, zero), (zero, one, None, zero, zero),
                     (u, zero, k, None, None), (u, one, k, None, zero)):
            status = status_word()
            want = qp.op_sample(x, *args, temperature_first=first, status=status)
            got = qp.op_sample(x, *(-a if a is zero else a for a in args), temperature_first=first, status=status)
            assert int(status) == 0 and (want[0] >= 0).all()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", [1, 5, 60])  # the last are streamed, and left to the clusters
@pytest.mark.parametrize("V,m,tail", [(152064, 0.69, 13.51), (152631, 0.69, 13.502)])
def test_a_nucleus_among_weights_of_a_few_units(qp, rows, V, m, tail):
    """One token, and all others at `tail` units of the row's fixed point, which count for 14: a little more than their share of what top_p = 1 - 2^-24
    leaves out, while `tail` is a little less.  A beginning of the others is left beside the first, by ids; of a streamed row, whose blocks sum up
    `tail` itself, the first alone may be left as well."""
    big = V // 2
    W = math.exp(m - math.floor(m / math.log(2)) * math.log(2)) * 2.0 ** (62 - 18)
    x = torch.full((rows, V), m + math.log(tail / W), device="cuda")
    x[:, big] = m
    units = math.exp(float(x[0, 0]) - float(x[0, big])) * W
    assert 13.5 < units - 2.0 ** -20 and units + 2.0 ** -20 < 14
    whole = W + 14 * (V - 1)
    n = math.ceil((14 * (V - 1) - whole * 2.0 ** -24) / 14)  # tokens left beside the first
    assert 0 < n < big
    p = torch.full((rows,), 1 - 2.0 ** -24, device="cuda")
    for u in (0.0, 2.0 ** -33, 2.0 ** -32, 2.0 ** -31, 2.0 ** -20, 0.5, 1 - 2.0 ** -24):
        token, logprob = qp.op_sample(x, torch.full((rows,), u, device="cuda"), None, None, p)
        want = u * (W + 14 * n) / 14  # of the others, 14 units each
        want = int(want) if want < n else big
        for r in range(rows):
            assert abs(int(token[r]) - want) <= 1 or rows == 60 and int(token[r]) == big, (u, int(token[r]), want)
            share = 1.0 if int(token[r]) == big else units / W
            close(logprob[r:r + 1], torch.tensor([math.log(share)], dtype=torch.float64, device="cuda"), 2.0 ** -22 + 2.0 ** -23 * abs(math.log(share)))


@pytest.mark.parametrize("rows,V", [(15000, 151936), (290001, 7501)])  # streamed, and kept by clusters
def test_logits_past_32_bits(qp, rows, V):
    """More than 2^31 logits: the rows of one call are those of calls on parts of them."""
    from test_gpu_sample import by_definition
    assert rows * V > 2 ** 31
    g = gen(9)
    x = torch.empty(rows, V, device="cuda").normal_(0, 3, generator=g)
    u = torch.rand(rows, generator=g, device="cuda")
    kinds = torch.arange(rows, device="cuda") % 4
    temp, k = torch.where(kinds == 0, 0.0, 0.8), torch.where(kinds == 1, 50, 0).to(I32)
    p = torch.where(kinds == 2, 0.9, 1.0)
    status = status_word()
    token, logprob = qp.op_sample(x, u, temp, k, p, status=status)
    assert int(status) == 0
    part = (rows + 5) // 6 // 4 * 4  # (the same addresses modulo 16)
    for at in range(0, rows, part):
        s = slice(at, min(at + part, rows))
        if V > 100000 and s.stop - at < 1000:
            continue  # (so few are kept)
        got = qp.op_sample(x[s], u[s], temp[s], k[s], p[s])
        assert torch.equal(got[0], token[s]) and torch.equal(got[1], logprob[s])
    edge = 2 ** 31 // V
    for r in (0, edge - 1, edge, edge + 1, rows - 3, rows - 2, rows - 1):
        want, _, near = by_definition(x[r], float(u[r]), float(temp[r]), int(k[r]), float(p[r]))
        assert near or int(token[r]) == want
