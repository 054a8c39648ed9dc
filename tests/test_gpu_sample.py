"""The next token of logits rows on the GPU against its definition in 64 bits.

Tokens are equal, but where the random number, or top_p, lies within NEAR of a border
of the 64-bit sums: weights are held to 2^-31, so a share of the whole is off by 2^-30
at most, and the 64-bit sums by far less (a gap of 0 among them may be one of 2^-54).
Where both sides' sums are whole numbers, as with equal logits, the tokens still agree."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_batch import BF16, F16, F32, I32, close, dev, gen, status_word  # noqa: E402

NEAR = 2.0 ** -30
INF = math.inf


@pytest.fixture(scope="module")
def qp():
    import quantized_transformer_prefill_gb300 as qp
    qp.lib()
    return qp


def by_definition(x, u, temp=1.0, k=0, p=1.0, floor=0.0, first=False):
    """(token, its log probability, whether a border is near) of one row."""
    x = x.double()
    at = torch.nonzero(x > -INF)[:, 0]
    if not len(at):
        return -1, -INF, False
    if temp == 0:
        return int(torch.nonzero(x == x.max())[0, 0]), 0.0, False
    sharp = temp if first else 1.0
    order = at[torch.sort(x[at], descending=True, stable=True).indices]
    if k > 0:
        order = order[:k]
    near = False
    w = torch.exp((x[order] - x[order[0]]) / sharp)
    n = len(order)
    if p < 1:
        before = w.cumsum(0) - w
        n = max(1, int((before < p * w.sum()).sum()))
        gap = ((before - p * w.sum()).abs() / w.sum()).min()
        near = float(gap) < NEAR
    order, w = order[:n], w[:n]
    if floor > 0:
        order = order[w >= floor * w[0]]
    order = order[(x[order] - x[order[0]]) / temp >= -60 * math.log(2)]
    left = order.sort().values
    w = torch.exp((x[left] - x[order[0]]) / temp)
    mass = w.cumsum(0)
    i = min(int((mass <= u * mass[-1]).sum()), len(left) - 1)
    gap = (mass / mass[-1] - u).abs().min()
    near |= float(gap) < NEAR and len(left) > 1
    top = w[i] / mass[-1]
    rest = (mass[-1] - w[i]) / mass[-1]
    logp = math.log1p(-float(rest)) if float(top) > 0.5 else float((x[left[i]] - x[order[0]]) / temp) - math.log(float(mass[-1]))
    return int(left[i]), logp, near


def check(qp, x, u, temp=None, k=None, p=None, floor=None, first=False):
    """One call on all rows against the definition, row by row."""
    rows = x.shape[0]
    f32 = lambda v: None if v is None else torch.tensor(v, dtype=F32, device="cuda")  # noqa: E731
    t_u, t_temp, t_p, t_floor = (f32(v) for v in (u, temp, p, floor))
    t_k = None if k is None else dev(k)
    status = status_word()
    token, logprob = qp.op_sample(x, t_u, t_temp, t_k, t_p, t_floor, temperature_first=first, status=status)
    assert int(status) == 0
    got, want, unsure = [], [], 0
    for r in range(rows):
        value = lambda t, default: default if t is None else t[r].item()  # noqa: B023, E731
        tok, logp, near = by_definition(x[r], float(t_u[r]), value(t_temp, 1.0), value(t_k, 0), value(t_p, 1.0), value(t_floor, 0.0), first)
        if near and (int(token[r]) != tok or abs(float(logprob[r]) - logp) > 1e-6):
            unsure += 1  # one token more or less is left, or the next one is drawn
            continue
        assert int(token[r]) == tok, (r, int(token[r]), tok)
        got.append(float(logprob[r])), want.append(logp)
    assert unsure <= 1 + rows // 100
    # a share is off by 2^-30 of the whole and the f32 result is rounded
    got, want = torch.tensor(got), torch.tensor(want, dtype=torch.float64)
    close(got, want, 2.0 ** -29 + 2.0 ** -23 * want.abs().nan_to_num(posinf=0, neginf=0))
    return token, logprob


def logits(g, rows, V, t, extra=0, masked=False):
    x = 2.5 * torch.randn(rows, V + extra, generator=g, device="cuda")
    likely = torch.randint(0, V, (rows, min(V, 6)), generator=g, device="cuda")
    x.scatter_(1, likely, 15 + 2 * torch.randn(likely.shape, generator=g, device="cuda"))
    if masked:
        x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < 0.5, -INF)
    return x.to(t)[:, :V]


SETTINGS = {
    "greedy": dict(temp=lambda r: 0.0),
    "plain": dict(temp=lambda r: 0.5 + 0.1 * (r % 10)),
    "k": dict(temp=lambda r: 0.8, k=lambda r: [1, 2, 5, 50, 200, 511][r % 6]),
    "k and p": dict(temp=lambda r: 0.7, k=lambda r: [1, 20, 64, 100][r % 4], p=lambda r: 0.3 + 0.06 * (r % 11)),
    "p": dict(temp=lambda r: 1.1, p=lambda r: [0.0, 0.1, 0.5, 0.9, 0.97, 0.999, 0.9999999][r % 7]),
    "min": dict(temp=lambda r: 1.3, floor=lambda r: [1.0, 0.3, 0.05, 0.001, 1e-7][r % 5]),
    "large k": dict(temp=lambda r: 1.5, k=lambda r: [513, 1000, 1024, 1025, 3000, 100000][r % 6], p=lambda r: 1.0 if r % 3 else 0.95),
    "hot": dict(temp=lambda r: 4.0 + r, p=lambda r: 0.99, floor=lambda r: 1e-9),
    "all": dict(temp=lambda r: 0.9, k=lambda r: 40 + r, p=lambda r: 0.95, floor=lambda r: 0.02),
    "each its own": dict(temp=lambda r: [0.0, 0.2, 1.0, 3.0][r % 4], k=lambda r: [0, 50, 0, 2000, -1][r % 5], p=lambda r: [1.0, 0.9, 2.0][r % 3],
                         floor=lambda r: [0.0, 0.1][r % 2]),
}


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("V,extra", [(1, 0), (2, 1), (33, 0), (1000, 7), (1025, 3), (5000, 0), (32001, 5), (151936, 0)])
@pytest.mark.parametrize("kind", list(SETTINGS))
def test_sample(qp, t, V, extra, kind):
    rows = 13
    g = gen(V + len(kind))
    x = logits(g, rows, V, t, extra, masked=V % 2 == 1 and V > 2)
    u = torch.rand(rows, generator=g, device="cuda").tolist()
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    settings = {name: [f(r) for r in range(rows)] for name, f in SETTINGS[kind].items()}
    for first in (False, True):
        check(qp, x, u, first=first, **settings)


@pytest.mark.parametrize("t,rows,V", [(F32, 52, 151936), (BF16, 130, 150001), (F16, 400, 40000)])
@pytest.mark.parametrize("kind", list(SETTINGS))
def test_sample_streamed_rows(qp, t, rows, V, kind):
    """More rows than their clusters fit the GPU: they are streamed."""
    g = gen(V + rows + len(kind))
    x = logits(g, rows, V, t, 3, masked=True)
    u = torch.rand(rows, generator=g, device="cuda").tolist()
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    x[rows // 2] = -INF
    assert qp.op_sample_workspace(x) is not None
    check(qp, x, u, first=kind in ("p", "all"), **{name: [f(r) for r in range(rows)] for name, f in SETTINGS[kind].items()})


def test_sample_borders_between_plateaus(qp):
    """top_p next to the share of a plateau of many equal logits, and a k next to its length: the border is one of two values
    that both keep more tokens than a list holds."""
    for V, rows in ((6000, 9), (151936, 9), (151936, 60)):
        x = torch.zeros(rows, V, device="cuda")
        x[:, 1::2] = 0.75
        upper = (V // 2) * math.exp(0.75)
        share = upper / (upper + (V - V // 2))
        p = [float(torch.tensor(share, dtype=F32)) + d * 2.0 ** -24 for d in (-40, -2, -1, 0, 1, 2, 40, -4000, 4000)]
        u = [0.1 * r for r in range(9)]
        for k in (None, [V // 2, V // 2 + 1, V // 2 - 1, 3000, V - 1, 0, 1, 2, V // 2]):
            settings = dict(p=(p * 7)[:rows]) if k is None else dict(k=(k * 7)[:rows], p=([1.0, 0.5, 0.9] * 20)[:rows])
            check(qp, x, (u * 7)[:rows], **settings)


@pytest.mark.parametrize("rows", [300, 5000])
def test_sample_many_rows(qp, rows):
    g = gen(rows)
    x = logits(g, rows, 4096 if rows < 1000 else 257, F32, 3)
    u = torch.rand(rows, generator=g, device="cuda").tolist()
    check(qp, x, u, temp=[0.5 + r % 7 / 5 for r in range(rows)], k=[r % 90 for r in range(rows)], p=[0.5 + r % 6 / 10 for r in range(rows)])


@pytest.mark.parametrize("t,V", [(F32, 200001), (F32, 700001), (BF16, 400003)])
def test_sample_rows_larger_than_shared_memory(qp, t, V):
    g = gen(V)
    x = logits(g, 7, V, t, 3)
    u = torch.rand(7, generator=g, device="cuda").tolist()
    check(qp, x, u, temp=[0.0, 1.0, 1.0, 0.7, 2.0, 2.0, 9.0], k=[0, 0, 50, 0, 5000, 0, 0], p=[1.0, 1.0, 1.0, 0.9, 0.9, 0.99, 0.9999])


def hard_row(kind, V):
    g = gen(17)
    x = torch.zeros(V, device="cuda")
    if kind == "two levels":
        x[::3] = 1.5
    elif kind == "few levels":
        x = torch.randint(0, 12, (V,), generator=g, device="cuda").float() / 4
    elif kind == "rising":
        x = torch.linspace(-30, 10, V, device="cuda")
    elif kind == "falling":
        x = torch.linspace(10, -30, V, device="cuda")
    elif kind == "one left":
        x.fill_(-INF)
        x[V // 2] = -7.0
    elif kind == "two left":
        x.fill_(-INF)
        x[V // 3], x[V - 1] = -7.0, -6.5
    elif kind == "none left":
        x.fill_(-INF)
    elif kind == "lowest":
        x.fill_(torch.finfo(F32).min)
        x[V // 4::V // 8] = torch.randn(len(x[V // 4::V // 8]), generator=g, device="cuda")
    elif kind == "all lowest":
        x.fill_(torch.finfo(F32).min)
    elif kind == "huge":
        x = 1e38 * torch.randn(V, generator=g, device="cuda")
    elif kind == "largest":
        x = (2e38 * torch.randn(V, generator=g, device="cuda")).nan_to_num()
    elif kind == "far":
        x = 70000 + torch.randn(V, generator=g, device="cuda")
    elif kind == "tiny":
        x = 1e-38 * torch.randn(V, generator=g, device="cuda")
    elif kind == "peak":
        x = torch.randn(V, generator=g, device="cuda")
        x[V // 2] = 40
    elif kind == "signed zeros":
        x[::2] = -0.0
    elif kind == "side by side":
        x = (torch.arange(V, device="cuda") % 97 + 1.0).mul(2.0 ** -20).add(3.0)
    return x


@pytest.mark.parametrize("kind", ["equal", "two levels", "few levels", "rising", "falling", "one left", "two left", "none left", "lowest", "all lowest",
                                  "huge", "largest", "far", "tiny", "peak", "signed zeros", "side by side"])
@pytest.mark.parametrize("V", [40, 5000, 151936])
def test_sample_hard_rows(qp, kind, V):
    """Every setting on rows of ties, plateaus, masks and extremes."""
    x = hard_row(kind, V)
    temp, k, p, floor, u = [], [], [], [], []
    for s in ((1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 20, 1.0, 0.0), (1.0, 2000, 1.0, 0.0), (1.0, 0, 0.5, 0.0), (2.0, 30, 0.75, 0.0), (1.0, 2500, 0.5, 0.0),
              (0.5, 0, 1.0, 0.25), (1.0, 3, 0.9, 0.5), (1e-6, 0, 1.0, 0.0), (1e6, 0, 0.5, 0.0), (1e6, 4000, 0.25, 0.0)):
        for v in (0.0, 0.4999, 0.5, 1 - 2.0 ** -24):
            for to, y in zip((temp, k, p, floor, u), (*s, v)):
                to.append(y)
    x = x.expand(len(u), V).contiguous()
    if x.max() == INF:  # of the huge rows the long ones go past f32: refused, and nothing else
        token, status = torch.full((len(u),), 77, dtype=I32, device="cuda"), status_word()
        qp.op_sample(x, torch.tensor(u, device="cuda"), torch.tensor(temp, device="cuda"), dev(k), out=(token, None), status=status)
        assert int(status) == -1 and (token == 77).all()
        return
    check(qp, x, u, temp=temp, k=k, p=p, floor=floor)


def test_sample_follows_the_distribution(qp):
    """Random numbers on a grid: every token comes as often as its probability says, to one step of the grid."""
    g = gen(1)
    n, V = 4000, 50
    x = torch.randn(1, V, generator=g, device="cuda").expand(n, V).contiguous()
    u = ((torch.arange(n, device="cuda") + 0.5) / n)
    token, logprob = qp.op_sample(x, u, torch.full((n,), 0.7, device="cuda"))
    share = torch.softmax(x[0].double() / 0.7, 0)
    count = torch.bincount(token.long(), minlength=V)
    assert ((count - n * share).abs() <= 1).all()
    close(logprob, torch.log(share)[token.long()], 1e-6)


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("t", [F32, BF16])
def test_sample_at_any_alignment(qp, t, offset):
    g = gen(offset)
    x = logits(g, 9, 5000, t, 13)[:, offset:offset + 4987]
    u = torch.rand(9, generator=g, device="cuda").tolist()
    for settings in (dict(), dict(k=[50] * 9), dict(p=[0.9] * 9), dict(temp=[0.0] * 9)):
        check(qp, x, u, **settings)


def test_sample_alone_and_in_a_batch(qp):
    """A row's token does not depend on the batch, whether it is kept or streamed; a call again gives the same bits."""
    g = gen(3)
    rows, V = 200, 50000
    x = logits(g, rows, V, F32)
    u = torch.rand(rows, generator=g, device="cuda")
    temp, k, p = torch.full((rows,), 1.2, device="cuda"), dev([r % 3 * 40 for r in range(rows)]), torch.full((rows,), 0.95, device="cuda")
    token, logprob = qp.op_sample(x, u, temp, k, p)
    for r in (0, 1, 2, 77, 199):
        one = qp.op_sample(x[r:r + 1], u[r:r + 1], temp[r:r + 1], k[r:r + 1], p[r:r + 1])
        assert torch.equal(one[0], token[r:r + 1])
        close(one[1], logprob[r:r + 1], 2.0 ** -28 + 2.0 ** -22 * logprob[r:r + 1].double().abs())
    for _ in range(3):
        again = qp.op_sample(x, u, temp, k, p)
        assert torch.equal(again[0], token) and torch.equal(again[1], logprob)


def test_sample_padding_and_refused_rows(qp):
    g = gen(4)
    for V, rows in ((60, 10), (5000, 10), (151936, 10), (151936, 60)):
        x = logits(g, rows, V, F32)
        u = torch.rand(rows, generator=g, device="cuda")
        want = qp.op_sample(x, u, torch.ones(rows, device="cuda"))
        bad = [("u", 1, -1.0, 0), ("u", 2, 1.0, -1), ("u", 3, math.nan, -1), ("temp", 4, -1.0, -1), ("temp", 5, math.nan, -1), ("temp", 6, 1e-7, -1),
               ("temp", 7, INF, -1), ("p", 1, -0.5, -1), ("p", 2, math.nan, -1), ("floor", 3, -0.1, -1), ("floor", 4, 1.5, -1), ("floor", 5, math.nan, -1),
               ("x", 6, math.nan, -1), ("x", 7, INF, -1), ("x", 8, -math.nan, -1)]
        for what, row, value, code in bad:
            a = dict(x=x.clone(), u=u.clone(), temp=torch.ones(rows, device="cuda"), p=torch.ones(rows, device="cuda"), floor=torch.zeros(rows, device="cuda"))
            if what == "x":
                a["x"][row, V // 3] = value
            else:
                a[what][row] = value
            out = (torch.full((rows,), 77, dtype=I32, device="cuda"), torch.full((rows,), 77.0, device="cuda"))
            status = status_word()
            qp.op_sample(a["x"], a["u"], a["temp"], None, a["p"], a["floor"], out=out, status=status)
            assert int(status) == code, (what, value)
            rest = [r for r in range(rows) if r != row]
            assert int(out[0][row]) == 77 and float(out[1][row]) == 77
            assert torch.equal(out[0][rest], want[0][rest]) and torch.equal(out[1][rest], want[1][rest])
    fresh = qp.op_sample(x, torch.full((rows,), -1.0, device="cuda"))
    assert (fresh[0] == -1).all() and (fresh[1] == 0).all()
    only = torch.empty(rows, dtype=I32, device="cuda")
    qp.op_sample(x, u, out=(only, None))
    assert torch.equal(only, want[0])


@pytest.mark.parametrize("rows,V", [(6, 30000), (60, 151936)])
def test_sample_streams_and_captured_graphs(qp, rows, V):
    """Two graphs captured on one side stream, replayed with other inputs, and calls at once on two streams."""
    g = gen(6)
    x = logits(g, rows, V, F32)
    u = torch.rand(rows, generator=g, device="cuda")
    k, p = dev([0, 50, 0, 700, 3, 0] * (rows // 6)), torch.tensor([1.0, 0.9, 0.9, 1.0, 1.0, 0.5] * (rows // 6), device="cuda")
    side = torch.cuda.Stream()
    graphs = []
    for i in range(2):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            qp.op_sample(x, u, None, k, p)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = qp.op_sample(x, u, None, k, p)
        graphs.append((graph, got))
    x.mul_(0.8)
    u.copy_(torch.rand(rows, generator=g, device="cuda"))
    torch.cuda.synchronize()
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = qp.op_sample(x, u, None, k, p)
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    other = torch.cuda.Stream()
    for s in (side, other):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(20):
        for s in (side, other):
            with torch.cuda.stream(s):
                got.append(qp.op_sample(x, u, None, k, p))
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, want))


def test_sample_workspaces(qp):
    """A workspace that is given serves calls of its shape whatever it holds; one that is too small is refused."""
    g = gen(8)
    x = logits(g, 60, 151936, F32)
    u = torch.rand(60, generator=g, device="cuda")
    p = torch.full((60,), 0.95, device="cuda")
    want = qp.op_sample(x, u, None, None, p)
    work = qp.op_sample_workspace(x)
    for fill in (0, 255, 77):
        work.fill_(fill)
        got = qp.op_sample(x, u, None, None, p, workspace=work)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(qp.MinferError, match="TOO_LARGE"):
        qp.op_sample(x, u, None, None, p, workspace=work[:-256])
    with pytest.raises(qp.MinferError, match="workspace"):
        qp.op_sample(x, u, None, None, p, workspace=work.int())
    assert qp.op_sample_workspace(x[:1]) is None


def test_rows_of_a_model_are_sampled(qp):
    """The rows of minfer_prefill_device_n go into op_sample, and the tokens' log probabilities are those of op_token_logprobs."""
    import synth
    from helpers import gpu_model
    cfg, w = synth.TINY, synth.WORKLOADS["tiny-32"]
    m = gpu_model(cfg)
    kv = m.kv(w.n_ctx)
    ids, pos = dev(w.ids().tolist()), dev(w.positions().tolist())
    x = torch.empty(32, cfg.n_vocab, device="cuda")
    torch.cuda.synchronize()
    assert m.prefill_device_n(kv, ids.data_ptr(), pos.data_ptr(), 32, 32, x.data_ptr()) == 0
    assert m.sync_status() == 0
    u = torch.rand(32, generator=gen(2), device="cuda")
    token, logprob = check(qp, x, u.tolist())
    close(logprob, qp.op_token_logprobs(x, token)[0].double(), 2e-6 * (1 + logprob.double().abs()))
    check(qp, x, u.tolist(), temp=[0.8] * 32, k=[50] * 32, p=[0.9] * 32, floor=[0.02] * 32)


def test_outputs_of_another_layout_are_refused(qp):
    x, u = torch.zeros(3, 50, device="cuda"), torch.rand(3, device="cuda")
    token, logprob = torch.zeros(3, dtype=I32, device="cuda"), torch.zeros(3, device="cuda")
    qp.op_sample(x, u, out=(token, logprob))
    for out, match in (((token.long(), logprob), "token"), ((token[:2], logprob), "token"), ((token, logprob.double()), "logprob"),
                       ((token, torch.zeros(4, device="cuda")), "logprob")):
        with pytest.raises(qp.MinferError, match=match):
            qp.op_sample(x, u, out=out)
    with pytest.raises(qp.MinferError, match="temperature"):
        qp.op_sample(x, u, torch.ones(2, device="cuda"))
    with pytest.raises(qp.MinferError, match="top_k"):
        qp.op_sample(x, u, None, torch.ones(3, device="cuda"))


@pytest.mark.parametrize("t,rows,V", [(F16, 400, 40000), (BF16, 130, 150001), (F32, 52, 151936), (BF16, 13, 151936)])
def test_sample_again_and_again(qp, t, rows, V):
    """The same call gives the same bits, however its warps happen to run: top-p borders in long tails, whose lists every CTA of
    a row's cluster adds to."""
    g = gen(V)
    x = logits(g, rows, V, t, 3, masked=True)
    u = torch.rand(rows, generator=g, device="cuda")
    p = torch.tensor([[0.5, 0.9, 0.97, 0.999, 0.9999999][r % 5] for r in range(rows)], device="cuda")
    temp = torch.full((rows,), 1.1, device="cuda")
    status = status_word()
    want = qp.op_sample(x, u, temp, top_p=p, temperature_first=True, status=status)
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        got = qp.op_sample(x, u, temp, top_p=p, temperature_first=True, status=status)
        off += (got[0] != want[0]).sum() + (got[1] != want[1]).sum()
    assert int(status) == 0 and int(off) == 0
