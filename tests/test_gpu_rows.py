"""moe_lora_permute / moe_lora_unpermute and their gradients against the float64
oracle, on layouts of moe_lora_align (whose pair_rows is checked first).

Bounds: a copy is exact; a sum of n fp32 terms in any order is off by at most
n * 2^-24 times the sum of the terms' magnitudes (every product and every
partial sum is rounded once, to half a step of 2^-23); the result's own rounding
adds eps / 2 of its type (bf16: 2^-8)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import rows_mx4_oracle as ro
from gpu_helpers import say
from moe_expert_layer_segment_amd import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def layout(T, k, E, block_m, seed, drop=0.0, loras=0):
    """A layout on the GPU and its pair_rows by the oracle; `drop`: share of pairs
    whose expert lives elsewhere (id -1 or past E)."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(T)]) if T else np.zeros((0, k))
    ids = ids.astype(np.int32)
    gone = rng.random(ids.shape) < drop
    ids[gone] = np.where(rng.random(ids.shape)[gone] < 0.5, -1, E + 3)
    slots = rng.integers(-1, max(loras, 1), size=max(T, 1)).astype(np.int32)
    en = torch.ones(loras, dtype=torch.int32, device="cuda") if loras else None
    al = binding.moe_lora_align(torch.from_numpy(ids).cuda(), torch.from_numpy(slots).cuda(), en, E,
                                loras, block_m, pair_rows=True)
    torch.cuda.synchronize()
    pr = ro.pair_rows_of(al["sorted_pair_ids"][:al["capacity"]].cpu().numpy(), T * k)
    if T:
        assert np.array_equal(al["pair_rows"].cpu().numpy(), pr)
        assert np.array_equal(pr >= 0, ~gone.reshape(-1))
    return al, pr


CASES = [  # T, k, E, block_m, hidden, dropped share, adapter slots
    (1, 1, 1, 16, 32, 0.0, 0),
    (1, 8, 16, 16, 2048, 0.0, 0),
    (64, 8, 128, 16, 2048, 0.0, 3),
    (37, 3, 5, 32, 1001, 0.0, 0),
    (130, 2, 4, 64, 1, 0.0, 0),
    (57, 6, 8, 16, 2056, 0.8, 2),
    (9, 9, 12, 16, 8200, 0.3, 0),
    (11, 2, 3, 16, 77, 1.0, 0),      # no pair has a row
    (300, 17, 32, 128, 130, 0.1, 0),
]
IDS = [f"T{c[0]}k{c[1]}E{c[2]}b{c[3]}H{c[4]}drop{c[5]}" for c in CASES]


def test_align_without_pair_rows_is_unchanged():
    """The other outputs of align do not depend on whether pair_rows is asked for."""
    rng = np.random.default_rng(3)
    ids = torch.from_numpy(rng.integers(0, 9, size=(200, 3)).astype(np.int32)).cuda()
    slots = torch.from_numpy(rng.integers(-1, 2, size=200).astype(np.int32)).cuda()
    en = torch.ones(2, dtype=torch.int32, device="cuda")
    a = binding.moe_lora_align(ids, slots, en, 9, 2, 16)
    b = binding.moe_lora_align(ids, slots, en, 9, 2, 16, pair_rows=True)
    assert "pair_rows" not in a
    for n in ("sorted_pair_ids", "tile_expert", "tile_lora", "expert_tile_offsets", "num_rows_padded"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "u8"])
def test_permute(case, dtype):
    T, k, E, bm, H, drop, loras = case
    say(f"permute {case} {dtype}")
    al, pr = layout(T, k, E, bm, 11, drop, loras)
    g = torch.Generator().manual_seed(5)
    if dtype == "u8":
        x = torch.randint(0, 256, (T, H), generator=g, dtype=torch.uint8).cuda()
        mark = torch.full((al["capacity"], H), 0xAB, dtype=torch.uint8, device="cuda")
    else:
        x = torch.randn(T, H, generator=g).to(DT[dtype]).cuda()
        x[0, 0] = float("inf")       # values are copied, whatever they are
        mark = torch.full((al["capacity"], H), 7.5, dtype=DT[dtype], device="cuda")
    out = binding.moe_lora_permute(x, al, k, out=mark.clone())
    torch.cuda.synchronize()
    ref, written = ro.permute(x.float().cpu().numpy(), pr, k, al["capacity"])
    used = int(al["num_rows_padded"].cpu()[0])
    got = out.float().cpu().numpy()
    assert np.array_equal(got[:used], ref[:used])
    assert not written[used:].any()
    assert torch.equal(out[used:], mark[used:]), "rows behind the last bucket were written"


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_unpermute_and_gradients(case, dtype, out):
    T, k, E, bm, H, drop, loras = case
    say(f"unpermute {case} {dtype}->{out}")
    al, pr = layout(T, k, E, bm, 12, drop, loras)
    cap, used = al["capacity"], int(al["num_rows_padded"].cpu()[0])
    g = torch.Generator().manual_seed(6)
    rows = torch.randn(cap, H, generator=g).to(DT[dtype]).cuda()
    # rows without a pair are never read
    dead = np.ones(cap, dtype=bool)
    dead[pr[pr >= 0]] = False
    rows[torch.from_numpy(dead).cuda()] = float("nan")
    w = torch.randn(T, k, generator=g).cuda()
    w.view(-1)[torch.from_numpy(pr < 0).cuda()] = float("nan")
    dy = torch.randn(T, H, generator=g).to(DT[out]).cuda()

    r64, w64, dy64 = np64(rows), np64(w), np64(dy)
    half = HALF[DT[out]]
    # y, with and without weights; the gradient of permute is the latter
    for weights, wn in ((w, w64), (None, None)):
        y = binding.moe_lora_unpermute(rows, al, k, weights, out_dtype=DT[out])
        ref, mag = ro.unpermute(r64, pr, k, wn)
        assert np.all(np.abs(np64(y) - ref) <= k * 2.0 ** -24 * mag * (1 + half) + half * np.abs(ref))
    dx = binding.moe_lora_permute_backward(rows, al, k, out_dtype=DT[out])
    assert torch.equal(dx, y)

    mark = torch.full((cap, H), -3.25, dtype=DT[dtype], device="cuda")
    d_rows, d_w = binding.moe_lora_unpermute_backward(dy, rows, al, k, w, d_rows=mark.clone())
    torch.cuda.synchronize()
    ref, ref_w, mag_w = ro.unpermute_backward(dy64, r64, pr, k, w64, cap)
    got = np64(d_rows)
    hr = HALF[DT[dtype]]
    # the product's own rounding, then the rows' type
    assert np.all(np.abs(got[:used] - ref[:used]) <= (2.0 ** -24 * (1 + hr) + hr) * np.abs(ref[:used]))
    assert torch.equal(d_rows[used:], mark[used:])
    # H products in fp32, in whatever grouping
    assert np.all(np.abs(np64(d_w) - ref_w) <= (H + 1) * 2.0 ** -24 * mag_w)
    # without d_weights the rows are not needed
    again, none = binding.moe_lora_unpermute_backward(dy, None, al, k, w, rows_dtype=DT[dtype],
                                                      d_rows=mark.clone())
    assert none is None and torch.equal(again, d_rows)
    # without weights d_rows is the copy
    ones, none = binding.moe_lora_unpermute_backward(dy, None, al, k, rows_dtype=DT[dtype],
                                                     d_rows=mark.clone())
    copy = binding.moe_lora_permute(dy.to(DT[dtype]), al, k, out=mark.clone())
    assert none is None and torch.equal(ones, copy)


def test_gradients_against_differences():
    """Directional differences of the fp32 forward.  y is linear in rows and in the
    weights, so the central difference over a step of 1 has no truncation error;
    what is left is the rounding of the two forwards and of the sums, at most
    (k + 2) * 2^-24 of the magnitudes each, 4 (k + 2) * 2^-24 with the loss's sum
    taken in float64."""
    T, k, E, H = 41, 4, 6, 520
    al, pr = layout(T, k, E, 16, 21, 0.2)
    cap = al["capacity"]
    g = torch.Generator().manual_seed(9)
    mk = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    rows, w, dy, vr, vw, x, vx = (mk(cap, H), mk(T, k), mk(T, H), mk(cap, H), mk(T, k), mk(T, H),
                                  mk(T, H))
    d_rows, d_w = binding.moe_lora_unpermute_backward(dy, rows, al, k, w,
                                                      d_rows=torch.zeros(cap, H, device="cuda"))
    loss = lambda r, ww: (np64(dy) * np64(binding.moe_lora_unpermute(r, al, k, ww))).sum()  # noqa: E731
    scale = 4 * (k + 2) * 2.0 ** -24
    for got, diff, mag in (
            ((np64(d_rows) * np64(vr)).sum(), (loss(rows + vr, w) - loss(rows - vr, w)) / 2,
             (np.abs(np64(dy)) * ro.unpermute(np.abs(np64(rows)) + np.abs(np64(vr)), pr, k,
                                              np.abs(np64(w)))[0]).sum()),
            ((np64(d_w) * np64(vw)).sum(), (loss(rows, w + vw) - loss(rows, w - vw)) / 2,
             (np.abs(np64(dy)) * ro.unpermute(np.abs(np64(rows)), pr, k,
                                              np.abs(np64(w)) + np.abs(np64(vw)))[0]).sum())):
        say(f"  differences: {got:.6f} {diff:.6f}")
        # d_weights sums H products, hence H / k more roundings there
        assert abs(got - diff) <= scale * (1 + H / k) * mag
        assert abs(diff) > 1e-3 * abs(mag) ** 0.5
    # permute and its gradient are transposes of one another
    c = mk(cap, H)
    used = int(al["num_rows_padded"].cpu()[0])
    fwd = (np64(c)[:used] * np64(binding.moe_lora_permute(vx, al, k))[:used]).sum()
    back = (np64(binding.moe_lora_permute_backward(c, al, k)) * np64(vx)).sum()
    mag = (ro.unpermute(np.abs(np64(c)), pr, k)[0] * np.abs(np64(vx))).sum()
    assert abs(fwd - back) <= k * 2.0 ** -24 * mag


def test_unaligned_pointers_and_long_rows():
    """Element-aligned views take the narrow path and give the same values."""
    T, k, E, H = 23, 2, 4, 264
    al, pr = layout(T, k, E, 16, 31)
    cap, used = al["capacity"], int(al["num_rows_padded"].cpu()[0])
    for dt in (torch.bfloat16, torch.float32, torch.uint8):
        mk = (lambda n: torch.randint(0, 255, (n,), device="cuda", dtype=dt)) if dt == torch.uint8 \
            else (lambda n: torch.randn(n, device="cuda").to(dt))
        x = mk(T * H + 1)[1:].view(T, H)
        out = mk(cap * H + 3)[3:].view(cap, H)
        binding.moe_lora_permute(x, al, k, out=out)
        ref = binding.moe_lora_permute(x.clone(), al, k)
        assert torch.equal(out[:used], ref[:used])
        if dt == torch.uint8:
            continue
        w = torch.randn(T, k, device="cuda")
        y = binding.moe_lora_unpermute(out, al, k, w, y=mk(T * H + 1)[1:].view(T, H))
        assert torch.equal(y, binding.moe_lora_unpermute(out.clone(), al, k, w))
        dr, dw = binding.moe_lora_unpermute_backward(x, out, al, k, w, d_rows=mk(cap * H + 1)[1:].view(cap, H))
        dr2, dw2 = binding.moe_lora_unpermute_backward(x.clone(), out.clone(), al, k, w)
        assert torch.equal(dr[:used], dr2[:used])
        # the same products, grouped over threads in another way
        bound = (H + 1) * 2.0 ** -23 * ro.unpermute_backward(
            np64(x), np64(out), pr, k, np64(w), cap)[2]
        assert np.all(np.abs(np64(dw) - np64(dw2)) <= bound)


def test_empty_batch():
    al, _ = layout(0, 2, 4, 16, 1)
    x = torch.zeros(0, 64, device="cuda")
    assert binding.moe_lora_permute(x, al, 2).shape == (0, 64)
    rows = torch.zeros(0, 64, device="cuda")
    w = torch.zeros(0, 2, device="cuda")
    assert binding.moe_lora_unpermute(rows, al, 2, w).shape == (0, 64)
    d, dw = binding.moe_lora_unpermute_backward(x, rows, al, 2, w)
    assert d.shape == (0, 64) and dw.shape == (0, 2)


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 4 GiB: 8192 wide bf16 rows, more than 2^31 elements."""
    T, k, E, H = 70000, 4, 8, 8192
    say("rows past 4 GiB")
    ids = (torch.arange(T, device="cuda").view(-1, 1) + torch.arange(k, device="cuda")) % E
    al = binding.moe_lora_align(ids.int(), torch.full((T,), -1, dtype=torch.int32, device="cuda"),
                                None, E, 0, 16, pair_rows=True)
    assert al["capacity"] * H > 1 << 31
    x = (torch.arange(T, device="cuda") % 251).bfloat16().view(-1, 1).expand(T, H).contiguous()
    rows = binding.moe_lora_permute(x, al, k)
    at = torch.tensor([0, T // 2, T - 1], device="cuda")
    pr = al["pair_rows"].view(T, k)
    for j in range(k):
        assert torch.equal(rows[pr[at, j].long()], x[at])
    w = torch.full((T, k), 0.25, device="cuda")
    assert torch.equal(binding.moe_lora_unpermute(rows, al, k, w), x)
    dr, dw = binding.moe_lora_unpermute_backward(x, rows, al, k, w)
    assert torch.equal(dr[pr[at, 0].long()], x[at] * 0.25)
    # sums of at most 251^2 * 8192 < 2^29 over equal terms: within 8192 roundings
    ref = (x[:, 0].double() ** 2 * H).view(-1, 1).expand(T, k)
    assert bool(((dw.double() - ref).abs() <= 8192 * 2.0 ** -24 * ref).all())


def test_streams_and_graph():
    """On a side stream, and captured: replays equal the eager results, with eager
    calls and new inputs between them."""
    T, k, E, H = 77, 4, 6, 1024
    al, _ = layout(T, k, E, 16, 41, 0.1)
    cap = al["capacity"]
    x, dy = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(T, k, device="cuda")
    rows, d_rows = (torch.zeros(cap, H, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw = torch.empty_like(w)

    def step():
        binding.moe_lora_permute(x, al, k, out=rows)
        binding.moe_lora_unpermute(rows, al, k, w, y=y)
        binding.moe_lora_unpermute_backward(dy, rows, al, k, w, d_rows=d_rows, d_weights=dw)
        binding.moe_lora_permute_backward(d_rows, al, k, dx=dx)
        return [t.clone() for t in (rows, y, d_rows, dw, dx)]

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(T, H, device="cuda"))
        want = step()
        for t in (rows, y, d_rows, dw, dx):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (rows, y, d_rows, dw, dx))), i
