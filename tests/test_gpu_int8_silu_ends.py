"""SiLU behind the integer products at the ends of fp32, where a gate's scaled exponent and its
correction leave fp32 long before SiLU itself does.

The tolerance is that of the products elsewhere: 4 * 2^-23 of the value (the exponential and the
reciprocal a step each; the exponent's correction, the sum and two products half a step each) and
the output type's rounding; SiLU below 2^-119 of a finite gate may be 0."""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from test_gpu_int8 import HALF, TINY, np64, product, silu64

pytestmark = pytest.mark.gpu

MAX = float(torch.finfo(torch.float32).max)


def ones(M, N, K):
    """Rows and columns whose sums are 1: y is the product of the scales."""
    x = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    w = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    x[:, 0] = 1
    w[:, 0] = 1
    return x, w


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("M,K", [(1, 16), (40, 528), (4160, 16), (4160, 528)])   # streamed, and by tiles
def test_silu_at_the_ends(M, K, dt):
    say(f"silu at the ends {M} {K} {dt}")
    half = 512
    size = torch.logspace(-30, np.log10(MAX) - 1e-4, half // 2 - 6, dtype=torch.float64).float()
    ends = torch.tensor([2.3e38, 2.37e38, 2.5e38, 3e38, MAX, 87.0])
    gate = torch.cat((size, ends, -size, -ends))
    x, w = ones(M, 2 * half, K)
    ws = torch.cat((gate, torch.full((half,), 0.5))).cuda()
    out = np64(product(x, torch.ones(M, device="cuda"), w, ws, silu=True, dt=dt))
    with np.errstate(over="ignore"):
        ref, up = silu64(ws.cpu().numpy().reshape(1, -1))
    tol = (4 * 2.0 ** -23 + HALF[dt]) * np.abs(ref) + 128 * TINY * (up + 1)
    assert not np.isnan(out).any()
    assert (np.abs(out - ref) <= tol).all()


@pytest.mark.parametrize("M,K", [(3, 16), (4160, 528)])
def test_silu_of_infinities(M, K):
    """SiLU(inf) is inf, of an infinite scale and of scales whose product leaves fp32; of -inf the
    formula has no value, and gives NaN."""
    say(f"silu of infinities {M} {K}")
    x, w = ones(M, 96, K)
    xs = torch.ones(M, device="cuda")
    xs[1] = 1e30                              # and gates of 1e30, of 1e50
    ws = torch.ones(96, device="cuda")
    ws[5], ws[6], ws[7], ws[8] = float("inf"), 1e20, float("nan"), -float("inf")
    out = product(x, xs, w, ws, silu=True, dt=torch.float32)
    want = torch.full((M, 48), 1 / (1 + np.exp(-1.0)), device="cuda")
    want[:, 6] = 1e20
    want[1] = want[:, 5] = float("inf")
    want[:, 7:9] = float("nan")
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.isinf(), want.isinf())
    some = want.isfinite()
    assert bool(((out - want).abs()[some] <= 5 * 2.0 ** -23 * want[some]).all())
