"""The balance loss and its gradient where probabilities, counts or differences are delicate: NaN
in any lane, logits far below the largest, one expert far above the others,
even counts, counts past 2^24."""
import numpy as np
import pytest
import torch

from oracle import int8_balance_oracle as ib
from gpu_helpers import say
from moe_expert_layer_segment_amd import binding
from test_gpu_balance import D, HALF, TINY, np64

pytestmark = pytest.mark.gpu


def gradient(logits, counts, n=None, k=1, d_loss=None):
    """d_logits for given counts, as a rank of a larger batch has them."""
    counts = torch.as_tensor(counts, dtype=torch.int32).cuda()
    n = logits.shape[0] if n is None else n
    stats = dict(counts=counts, num_valid=torch.tensor([n], dtype=torch.int32).cuda(), top_k=k)
    return binding.moe_lora_balance_loss_backward(d_loss, logits, stats, out_dtype=torch.float32)


def differences(logits, counts, n=None, k=1):
    """(gradient, size): g p_e sum_i p_i (c_e - c_i) and g p_e sum_i p_i |c_e - c_i| in float64.
    Probabilities that are off by a factor 1 + d each leave the gradient off by 2 |d| of the size."""
    l64 = np64(logits)
    p, c = ib.softmax(l64), np.asarray(counts, dtype=np.float64)
    T, E = l64.shape
    n = T if n is None else n
    g = E / (float(n) ** 2 * k)
    diff = c[:, None] - c[None, :]
    return g * p * (p @ diff.T), g * p * (p @ np.abs(diff).T)



# ---------------------------------------------------------------------------
# NaN
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("off", ["lower", "upper", "all", "none"])
@pytest.mark.parametrize("E", [64, 100, 256, 1000])
def test_nan_at_every_expert(E, off):
    """A row with a NaN anywhere is NaN as a whole, whichever of its experts are switched off."""
    say(f"nan {E} {off}")
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(E, E, generator=g)
    half = E // 2
    if off != "none":
        logits[:, {"lower": slice(half), "upper": slice(half, E), "all": slice(E)}[off]] = float("-inf")
    logits.fill_diagonal_(float("nan"))
    logits = logits.cuda()
    d = gradient(logits, torch.randint(0, 50, (E,), generator=g))
    assert bool(d.isnan().all())
    ids = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for t in {0, 1, half - 1, half, half + 1, half + half // 2, E - 1}:
        stats = binding.moe_lora_balance_loss(logits[t:t + 1], ids)
        assert bool(stats["mean_probs"].isnan().all()) and bool(stats["loss"].isnan().all()), t


# ---------------------------------------------------------------------------
# logits far below the largest
# ---------------------------------------------------------------------------
def far_rows(E, n, seed, below=86.0):
    """fp32 rows whose largest logit is small or negative, the others far below it."""
    g = torch.Generator().manual_seed(seed)
    top = 65 * torch.rand(n, 1, generator=g, dtype=torch.float64) - 60
    logits = top - 20 - (below - 20) * torch.rand(n, E, generator=g, dtype=torch.float64)
    at = torch.randint(0, E, (n, 1), generator=g)
    return logits.scatter(1, at, top).float().cuda()


@pytest.mark.parametrize("E", [64, 300, 1024])
def test_logits_far_below_a_negative_one(E):
    """Each probability of a token alone is within D of its value: the difference to the largest
    logit is taken to more digits than fp32 holds of it."""
    say(f"far below {E}")
    ids = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    logits = far_rows(E, 40, 2)
    p = ib.softmax(np64(logits))
    for t in range(40):
        mean = np64(binding.moe_lora_balance_loss(logits[t:t + 1], ids)["mean_probs"])
        assert (np.abs(mean - p[t]) <= (D + HALF[torch.float32]) * p[t] + TINY).all(), t


# ---------------------------------------------------------------------------
# differences of counts
# ---------------------------------------------------------------------------
def peaked_rows(E, n, seed):
    """Rows with one logit 15 to 30 above the others'."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(n, E, generator=g)
    at = torch.randint(0, E, (n, 1), generator=g)
    return logits.scatter(1, at, 15 + 15 * torch.rand(n, 1, generator=g)).cuda()


# what 64 bits leave of c_e - sum_i p_i c_i / sum_i p_i, of c: two sums of 16 terms in a lane and of six
# exchanges, a quotient and a difference: 46 half steps of 2^-53
LAST = 2.0 ** -47


@pytest.mark.parametrize("E", [2, 64, 200, 1024])
def test_gradient_of_peaked_rows(E):
    """Where one expert has all but a millionth of the probability its gradient is a difference of
    nearly equal numbers; what the rounding of probabilities leaves is of the size of the
    differences of counts alone, and rows add up to 0."""
    say(f"peaked rows {E}")
    g = torch.Generator().manual_seed(3)
    counts = torch.randint(1500, 2501, (E,), generator=g)
    logits = peaked_rows(E, 200, 4)
    d = np64(gradient(logits, counts))
    ref, size = differences(logits, counts)
    noise = LAST * E / 200.0 ** 2 * 2500
    tol = 2.01 * D * size + HALF[torch.float32] * (np.abs(ref) + 2.01 * D * size) + noise + TINY
    assert (np.abs(d - ref) <= tol).all()
    # each element is rounded twice (p, and the result)
    assert (np.abs(d.sum(1)) <= 2.01 * 2.0 ** -24 * np.abs(d).sum(1) + E * (noise + TINY)).all()


@pytest.mark.parametrize("E", [1, 2, 61, 64, 256, 1000])
def test_gradient_of_even_counts_is_zero(E):
    say(f"even counts {E}")
    for logits in (peaked_rows(E, 50, 5), torch.randn(50, E, generator=torch.Generator().manual_seed(6)).cuda()):
        d = np64(gradient(logits, [12345] * E))
        p = ib.softmax(np64(logits))
        assert (np.abs(d) <= LAST * 12345 * E / 50.0 ** 2 * p * (1 + D) + TINY).all()


@pytest.mark.parametrize("base", [1 << 24, (1 << 28) + 3, (1 << 31) - 2000])
@pytest.mark.parametrize("E", [8, 65, 512])
def test_counts_past_24_bits(E, base):
    """Counts summed over ranks differ by less than fp32 holds of them."""
    say(f"counts {E} {base}")
    g = torch.Generator().manual_seed(7)
    counts = base + torch.randint(0, 1000, (E,), generator=g)
    logits = torch.randn(60, E, generator=g).cuda()
    n = 1 << 26
    d = np64(gradient(logits, counts, n, 8))
    ref, size = differences(logits, counts, n, 8)
    noise = LAST * E / (float(n) ** 2 * 8) * base
    tol = 2.01 * D * size + HALF[torch.float32] * (np.abs(ref) + 2.01 * D * size) + noise + TINY
    assert (np.abs(d - ref) <= tol).all()


# ---------------------------------------------------------------------------
# probabilities
# ---------------------------------------------------------------------------
# A probability before it is rounded: in 2^f = 1 + f (ln 2 + f (c + f R(f))) R is fp32, two half steps of a
# number below 2^-4 and less than another from the steps before, times |f|^3 <= 1/8, of a result above 0.7,
# and what the series leaves out 2^-31: below 2^-29.  The sum of them is off by as much.
P = 2.0 ** -28


def test_probabilities_have_more_bits_than_fp32():
    """mean_probs of a token alone, the loss and the gradient are off by little more than their last
    rounding, down to the last numbers that fp32 has."""
    say("probabilities")
    ids = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    half = HALF[torch.float32] * (1 + P)
    for E in (7, 64, 256, 1024):
        near = torch.randn(40, E, generator=torch.Generator().manual_seed(8)).cuda()
        for logits in (near, 4 * near, far_rows(E, 40, 9, 110.0)):
            p = ib.softmax(np64(logits))
            for t in range(40):
                stats = binding.moe_lora_balance_loss(logits[t:t + 1], ids)
                assert (np.abs(np64(stats["mean_probs"]) - p[t]) <= (P + half) * p[t] + 2.0 ** -150).all()
                assert abs(float(stats["loss"].cpu()[0]) - E * p[t, 0]) <= (P + half) * E * p[t, 0] + 2.0 ** -150
            counts = torch.randint(0, 99, (E,), generator=torch.Generator().manual_seed(10))
            d, (ref, size) = np64(gradient(logits, counts)), differences(logits, counts)
            noise = LAST * E / 40.0 ** 2 * 99 * p
            assert (np.abs(d - ref) <= 2.01 * P * size + half * (np.abs(ref) + 2.01 * P * size) + noise + 2.0 ** -150).all()
