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
