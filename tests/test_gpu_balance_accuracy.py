"""The balance loss and its gradient where probabilities, counts or differences are delicate: NaN
in any lane, logits far below the largest."""
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
