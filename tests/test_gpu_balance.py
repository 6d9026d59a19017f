"""The router's balance loss and its gradient against the float64 oracle.

Counts are exact.  A probability is within D = 32 * 2^-24 of its value: the exponential is off
by two half steps at most, its correction and product by one each, a sum of up to 1024 of them
(16 in a lane and six exchanges) by 22, the reciprocal and the last product by one each: 28.
mean_probs and loss are sums of positive terms in 64 bits, so off by D and their last rounding.
The gradient g p (c - sum p c) is off by D of g p (|c - sum p c| + sum p c), and its last
rounding.  Probabilities below 2^-126 may be 0."""
import numpy as np
import pytest
import torch

from oracle import int8_balance_oracle as ib
from gpu_helpers import say
from moe_expert_layer_segment_amd import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
D = 32 * 2.0 ** -24
TINY = 2.0 ** -126


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def routed(T, E, k, dtype, seed, off=0):
    g = torch.Generator().manual_seed(seed)
    logits = 3 * torch.randn(T, E, generator=g) + torch.randn(E, generator=g)
    if off:
        logits[:, torch.randperm(E, generator=g)[:off]] = float("-inf")
    logits = logits.to(DT[dtype])
    ids = torch.topk(logits.float(), k, dim=1).indices.int() if T else torch.empty(0, k, dtype=torch.int32)
    return logits.cuda(), ids.cuda()


def check(logits, ids, mask=None, d_loss=None, out_dtype=None, stats=None):
    T, E = logits.shape
    if stats is None:
        stats = binding.moe_lora_balance_loss(logits, ids, mask)
    host = None if mask is None else mask.cpu().numpy()
    loss, counts, mean, n, _ = ib.balance_loss(np64(logits), ids.cpu().numpy(), host)
    assert np.array_equal(stats["counts"].cpu().numpy(), counts)
    assert int(stats["num_valid"].cpu()[0]) == n and stats["top_k"] == ids.shape[1]
    assert (np.abs(np64(stats["mean_probs"]) - mean) <= (D + HALF[torch.float32]) * mean + TINY).all()
    assert abs(float(stats["loss"].cpu()[0]) - loss) <= (D + HALF[torch.float32]) * loss + TINY * E
    g = None if d_loss is None else torch.tensor([d_loss], device="cuda")
    d = binding.moe_lora_balance_loss_backward(g, logits, stats, mask, out_dtype=out_dtype)
    ref, mag = ib.balance_loss_backward(1.0 if d_loss is None else float(np.float32(d_loss)), np64(logits),
                                        counts, n, ids.shape[1], host)
    assert d.dtype == (out_dtype or logits.dtype)
    tol = D * mag + HALF[d.dtype] * (np.abs(ref) + D * mag) + TINY * (1 + mag)
    assert (np.abs(np64(d) - ref) <= tol).all()
    return stats, d


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (3, 61, 6), (64, 128, 8), (256, 64, 2), (257, 65, 3),
                                   (300, 256, 8), (1000, 257, 4), (2049, 512, 8), (2500, 8, 2), (700, 1000, 5),
                                   (333, 1024, 16), (50, 1024, 70)])
def test_loss_and_gradient(T, E, k, dtype):
    say(f"balance {T} {E} {k} {dtype}")
    logits, ids = routed(T, E, k, dtype, 1)
    check(logits, ids)
    check(logits, ids, d_loss=-0.37, out_dtype=torch.float32)
    g = torch.Generator().manual_seed(2)
    mask = (torch.rand(T, generator=g) < 0.6).cuda()
    check(logits, ids, mask, 2.5, torch.bfloat16)
    check(logits, ids, mask.to(torch.uint8) * 200)


@pytest.mark.parametrize("T", [5, 400])
def test_masked_tokens_are_not_read(T):
    """What padding tokens hold reaches nothing; their gradient is 0."""
    logits, ids = routed(T, 40, 4, "f32", 3)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[2::5] = False
    clean, d = check(logits, ids, mask)
    logits2, ids2 = logits.clone(), ids.clone()
    logits2[~mask] = float("nan")
    ids2[~mask] = 1 << 30
    stats = binding.moe_lora_balance_loss(logits2, ids2, mask)
    d2 = binding.moe_lora_balance_loss_backward(None, logits2, stats, mask)
    assert all(torch.equal(stats[n], clean[n]) for n in ("loss", "counts", "mean_probs", "num_valid"))
    assert torch.equal(d, d2) and not bool(d2[~mask].any())


@pytest.mark.parametrize("T", [0, 1, 300])
def test_no_token_takes_part(T):
    logits, ids = routed(T, 9, 2, "f32", 4)
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    stats = binding.moe_lora_balance_loss(logits, ids, mask)
    assert not any(bool(stats[n].any()) for n in ("loss", "counts", "mean_probs", "num_valid"))
    d = binding.moe_lora_balance_loss_backward(None, logits, stats, mask)
    assert d.shape == (T, 9) and not bool(d.any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [30, 600])
def test_experts_switched_off(T, dtype):
    """-inf, the type's lowest value, rows of either alone, and very unlike logits."""
    logits, ids = routed(T, 70, 4, dtype, 5, off=20)
    logits[0] = float("-inf")
    logits[1] = torch.finfo(logits.dtype).min
    logits[2, ::2] = torch.finfo(logits.dtype).min
    logits[3] = torch.finfo(logits.dtype).min
    logits[3, 5] = torch.finfo(logits.dtype).max
    logits[4] = 80.0
    logits[5, :35] = -300.0
    stats, d = check(logits, ids)
    assert not bool(d[0].any())
    assert bool(d.isfinite().all())


@pytest.mark.parametrize("T", [20, 500])
def test_nan_and_infinity_are_not_hidden(T):
    for bad in (float("nan"), float("inf")):
        logits, ids = routed(T, 33, 3, "f32", 6)
        logits[7, 31] = bad
        stats = binding.moe_lora_balance_loss(logits, ids)
        assert bool(stats["loss"].isnan().all()) and int(stats["counts"].sum().cpu()) == 3 * T
        d = binding.moe_lora_balance_loss_backward(None, logits, stats)
        assert bool(d[7, 31].isnan()) and bool(d[torch.arange(T, device="cuda") != 7].isfinite().all())


@pytest.mark.parametrize("T", [40, 900])
def test_ids_of_other_ranks(T):
    """Ids outside [0, E) count nowhere; an id named twice by a token counts twice."""
    logits, ids = routed(T, 16, 4, "f32", 7)
    ids[::3, 0] = -1
    ids[1::3, 1] = 16
    ids[2::3, 2] = 1 << 30
    ids[5, 3] = ids[5, 1] = 11
    check(logits, ids)


def test_given_outputs_and_workspace():
    logits, ids = routed(700, 48, 3, "f32", 8)
    ref, _ = check(logits, ids)
    n = binding.moe_lora_balance_loss_workspace_bytes(700, 48)
    ws = torch.full((n,), 171, dtype=torch.uint8, device="cuda")
    out = dict(loss=torch.full((1,), 9.0, device="cuda"),
               counts=torch.full((48,), 9, dtype=torch.int32, device="cuda"),
               mean_probs=torch.full((48,), 9.0, device="cuda"),
               num_valid=torch.full((1,), 9, dtype=torch.int32, device="cuda"))
    for _ in range(3):   # nothing is left over from the call before
        got = binding.moe_lora_balance_loss(logits, ids, out=out, workspace=ws)
        assert all(got[n] is out[n] and torch.equal(got[n], ref[n]) for n in out)
    d = torch.full((700, 48), 5.0, device="cuda")
    assert binding.moe_lora_balance_loss_backward(None, logits, got, d_logits=d) is d
    assert torch.equal(d, binding.moe_lora_balance_loss_backward(None, logits, ref))


def test_ranks_of_a_batch():
    """Counts and numbers of tokens summed over two ranks: their gradients are the whole's."""
    logits, ids = routed(900, 24, 3, "f32", 9)
    whole = binding.moe_lora_balance_loss(logits, ids)
    d = binding.moe_lora_balance_loss_backward(None, logits, whole)
    parts = [(logits[:350].contiguous(), ids[:350].contiguous()), (logits[350:].contiguous(), ids[350:].contiguous())]
    stats = [binding.moe_lora_balance_loss(*p) for p in parts]
    both = dict(top_k=3, counts=stats[0]["counts"] + stats[1]["counts"],
                num_valid=stats[0]["num_valid"] + stats[1]["num_valid"])
    got = torch.cat([binding.moe_lora_balance_loss_backward(None, p[0], both) for p in parts])
    assert torch.equal(got, d)


def test_gradient_against_differences():
    """Along the gradient of length one the loss changes by its length times the step.  With
    counts fixed L is smooth: the difference of two losses 2 h apart is off by 2 (D + 2^-24) L / 2 h
    from rounding and h^2 / 6 of the third derivative, which p (1 - p) ... bounds by max
    |c| E / (n k) times the cube of the step's largest entry."""
    T, E, k = 6, 8, 2
    logits, ids = routed(T, E, k, "f32", 10)
    stats = binding.moe_lora_balance_loss(logits, ids)
    d = binding.moe_lora_balance_loss_backward(None, logits, stats)
    length = float(d.norm().cpu())
    step = d / length
    h = 0.05
    a, b = (float(binding.moe_lora_balance_loss((logits + s * h * step).contiguous(), ids)["loss"].cpu()[0])
            for s in (1, -1))
    c = E / (T * k) * float(stats["counts"].max().cpu())
    tol = 2 * (D + 2.0 ** -24) * a / (2 * h) + h * h / 6 * c * 6 * float(step.abs().max().cpu()) ** 3 + 2.0 ** -22 * length
    assert abs((a - b) / (2 * h) - length) <= tol and tol < 0.2 * length


class Balance(torch.autograd.Function):
    """How a training step has the loss."""

    @staticmethod
    def forward(ctx, logits, ids, mask):
        stats = binding.moe_lora_balance_loss(logits, ids, mask)
        ctx.save_for_backward(logits, mask)
        ctx.stats = stats
        return stats["loss"]

    @staticmethod
    def backward(ctx, d_loss):
        logits, mask = ctx.saved_tensors
        return binding.moe_lora_balance_loss_backward(d_loss.contiguous(), logits, ctx.stats, mask), None, None


def test_training_step():
    """router -> route -> loss with the rows' combine behind it, both gradients through autograd:
    the router's weights get those of the formulas in 64 bits."""
    T, E, k, H = 300, 12, 2, 40
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, H, generator=g).cuda()
    w = torch.nn.Parameter(torch.randn(E, H, generator=g).cuda() * H ** -0.5)
    mask = (torch.rand(T, generator=g) < 0.8).cuda()
    logits = x @ w.t()
    ids, _ = binding.moe_lora_route(logits.detach(), k)
    loss = 0.01 * Balance.apply(logits, ids, mask).sum()
    loss.backward()
    l64 = np64(logits)
    _, counts, _, n, _ = ib.balance_loss(l64, ids.cpu().numpy(), mask.cpu().numpy())
    ref, mag = ib.balance_loss_backward(float(np.float32(0.01)), l64, counts, n, k, mask.cpu().numpy())
    dw = ref.T @ np64(x)
    # fp32 sums of T products, and the gradient's own error
    tol = (T * 2.0 ** -24 + 2 * D) * (mag.T @ np.abs(np64(x))) + TINY
    assert (np.abs(np64(w.grad) - dw) <= tol).all()


def test_results_do_not_change():
    logits, ids = routed(5000, 100, 4, "f32", 12)
    first = binding.moe_lora_balance_loss(logits, ids)
    for _ in range(5):
        again = binding.moe_lora_balance_loss(logits, ids)
        assert all(torch.equal(first[n], again[n]) for n in ("loss", "counts", "mean_probs"))
