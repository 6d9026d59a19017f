"""Rows in expert order and MX4 products where a call's arguments, sizes or values
leave the ordinary: reused buffers, weights that are not finite, every variant of the
kernels, sizes past one launch.  Products are compared as in test_gpu_mx4, within its
bounds."""
import numpy as np
import pytest
import torch

from oracle import rows_mx4_oracle as ro
from gpu_helpers import say
from moe_expert_layer_segment_amd import binding
from test_gpu_mx4 import activations, check_product, np64, weights

pytestmark = pytest.mark.gpu


def empty_layout(T, k, E, block_m):
    """Buffers of moe_lora_align for up to T tokens, filled with what no layout holds."""
    cap = binding.moe_lora_align_capacity_rows(T, k, E, 0, block_m)
    i32 = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(sorted_pair_ids=i32(cap), tile_expert=i32(cap // block_m), tile_lora=i32(cap // block_m),
                expert_tile_offsets=i32(E + 1), num_rows_padded=i32(1), pair_rows=i32(T * k))


def some_ids(T, k, E, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()


def no_slots(T):
    return torch.full((max(T, 1),), -1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("bm", [16, 64])
def test_layout_in_buffers_of_a_larger_batch(kind, bm):
    """The results are those of a layout of the batch's own size: padding rows (NaN
    here) give zeros, and the rows sum up to the batch's tokens."""
    k, E, N, K = 2, 5, 96, 160
    out = empty_layout(300, k, E, bm)
    wc, ws, _ = weights(E, N, K, 31)
    for T in (300, 41, 1):
        say(f"larger buffers {kind} block_m {bm} T {T}")
        ids = some_ids(T, k, E, T)
        own = binding.moe_lora_align(ids, no_slots(T), None, E, 0, bm, pair_rows=True)
        al = binding.moe_lora_align(ids, no_slots(T), None, E, 0, bm, out=out, pair_rows=True)
        cap, used = al["capacity"], int(al["num_rows_padded"].cpu()[0])
        assert cap == own["capacity"] and al["num_pairs"] == T * k
        x, xs, _ = activations(cap, K, kind, 32)
        pad = al["sorted_pair_ids"][:cap] >= T * k
        (x if kind == "bf16" else xs)[pad] = float("nan") if kind == "bf16" else 255
        z, z2 = (binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=a, out_dtype=torch.float32)
                 for a in (al, own))
        assert torch.equal(z[:used], z2[:used]) and bool((z[:used][pad[:used]] == 0).all())
        w = torch.rand(T, k, device="cuda")
        y, y2 = (binding.moe_lora_unpermute(z, a, k, w) for a in (al, own))
        assert y.shape == (T, N) and torch.equal(y, y2)


def test_layout_reused_without_pair_rows():
    """Rows placed by a reused layout are those of its last batch."""
    T, k, E, H = 90, 2, 6, 64
    al = binding.moe_lora_align(some_ids(T, k, E, 1), no_slots(T), None, E, 0, 16, pair_rows=True)
    ids = some_ids(T, k, E, 2)
    binding.moe_lora_align(ids, no_slots(T), None, E, 0, 16, out=al)
    own = binding.moe_lora_align(ids, no_slots(T), None, E, 0, 16, pair_rows=True)
    x = torch.randn(T, H, device="cuda")
    used = int(own["num_rows_padded"].cpu()[0])
    assert torch.equal(al["pair_rows"], own["pair_rows"])
    assert torch.equal(binding.moe_lora_permute(x, al, k)[:used], binding.moe_lora_permute(x, own, k)[:used])


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("bm", [16, 32, 48, 64, 128, 192, 256])
@pytest.mark.parametrize("tokens", [9, 2000])
def test_padding_rows_beside_weights_that_are_not_finite(kind, bm, tokens):
    """Padding rows get zeros also where a weight is NaN (a scale byte of 255, as the
    quantisation gives it) or, beside bf16 x, past the largest finite value (codes of 4
    and 6 under 254); every other column of the rows that hold a pair keeps its bits."""
    k, E, N, K = 2, 5, 160, 544
    say(f"weights that are not finite {kind} block_m {bm} T {tokens}")
    al = binding.moe_lora_align(some_ids(tokens, k, E, 7), no_slots(tokens), None, E, 0, bm, pair_rows=True)
    used, M = int(al["num_rows_padded"].cpu()[0]), al["capacity"]
    live = (al["sorted_pair_ids"][:M] < tokens * k)[:used]
    assert not bool(live.all())
    wc, ws, _ = weights(E, N, K, 33)
    x, xs, _ = activations(M, K, kind, 34)
    bad = ws.clone()
    bad[:, 5, 3], bad[:, 90, K // 32 - 1] = 255, 254
    wc[:, 90, -1] = 0x77   # two sixes
    for silu in (False, True):
        y, clean = (binding.moe_lora_mx4_gemm(x, wc, w, x_scales=xs, align_out=al, silu_mul=silu,
                                              out_dtype=torch.float32)[:used] for w in (bad, ws))
        assert bool((y[~live] == 0).all())
        hit = [5, 90 - 80] if silu else [5, 90]
        assert bool(torch.isnan(y[live][:, 5]).all())
        keep = torch.ones(y.shape[1], dtype=torch.bool, device="cuda")
        keep[hit] = False
        assert torch.equal(y[:, keep], clean[:, keep])


# ---------------------------------------------------------------------------
# every variant of the product kernels
# ---------------------------------------------------------------------------
VARIANTS = [  # block_m (None: one weight for all rows), blocks or rows, N, K
    (16, 37, 1040, 1056), (16, 33, 48, 96), (16, 64, 512, 16416), (48, 13, 1040, 544), (16, 33, 48, 16416),
    (32, 33, 1040, 1056), (32, 33, 64, 160), (32, 64, 512, 16416), (96, 17, 1552, 288),
    (16, 17, 2016, 288), (32, 17, 2016, 160), (None, 1, 32784, 96), (None, 20, 32784, 96),
    (64, 2, 8176, 288), (64, 34, 256, 96), (64, 32, 512, 96), (64, 16, 1008, 16416),
    (None, 64, 16384, 96), (None, 40, 16368, 32),
    (None, 1, 48, 16416), (None, 20, 48, 16416), (None, 64, 48, 16416),
    (None, 1, 48, 16384), (None, 20, 48, 16384), (None, 64, 48, 16384),
    # more than 4096 tiles: the last round is not split
    (64, 258, 4112, 96), (64, 242, 4352, 128), (128, 260, 4112, 32), (256, 242, 4128, 128),
    (None, 61700, 4352, 32),
]


def variant(M, N, K, block_m, kind):
    """What launch_mx4_gemm takes: ("stream", 16-row blocks, 16-column blocks, waves, groups of
    rows in sixteens, scales in LDS) or ("tile", rows, last round split, scales by DMA)."""
    up = lambda a, b: -(-a // b)  # noqa: E731

    def takes(n):
        return block_m % n == 0 if block_m else M > n // 2

    def few(mb, nb, wide):
        groups = up(M, 16 * mb)
        full = groups * up(N, 16 * nb) >= 512
        return "stream", mb, nb if full else 2, 4 if full else wide, groups >= 32, K <= 16384

    if takes(64):
        if up(M, 64) * up(N, 256) <= 64:
            return few(4, 2, 8)
        rows = 256 if takes(256) else 128 if takes(128) else 64
        return "tile", rows, up(M, rows) * up(N, 256) <= 4096, kind == "bf16" and K % 128 == 0
    return few(2, 4, 8) if takes(32) else few(1, 4, 16)


@pytest.mark.parametrize("case", VARIANTS, ids=lambda c: f"b{c[0]}n{c[1]}N{c[2]}K{c[3]}")
@pytest.mark.parametrize("kind", ["bf16", "mx4"])
def test_variants(case, kind):
    """Blocks of any number of rows that hold a pair, against the oracle (of more than 2^24
    results a share of the rows, those at the borders of blocks and at the end among them)."""
    bm, n, N, K = case
    E, M = (3, bm * n) if bm else (1, n)
    say(f"variant {case} {kind}: {variant(M, N, K, bm, kind)}")
    g = torch.Generator().manual_seed(41)
    experts, live = torch.zeros(M, dtype=torch.long), torch.ones(M, dtype=torch.bool)
    al = None
    if bm:
        tiles = torch.randint(0, E, (n,), generator=g)
        tiles[-1] = -1
        experts = tiles.repeat_interleave(bm)
        fill = torch.randint(0, bm + 1, (n, 1), generator=g)
        fill[:3] = torch.tensor([[0], [bm], [1]])[:n]
        live = (torch.arange(bm) < fill).view(-1) & (torch.rand(M, generator=g) < 0.95)
        pairs = int(live.sum()) + 1
        sid = torch.full((M,), pairs, dtype=torch.int32)
        sid[live] = torch.randperm(pairs - 1, generator=g).int()
        al = dict(block_m=bm, tile_expert=tiles.int().cuda(), sorted_pair_ids=sid.cuda(),
                  pair_rows=torch.empty(pairs, dtype=torch.int32, device="cuda"))
    wc, ws, w64 = weights(E, N, K, 42)
    x, xs, x64 = activations(M, K, kind, 43)
    at = torch.arange(M)
    if M * N > 1 << 24:
        at = at[(at % 61 == 0) | (at % (bm or 256) < 2) | (at >= M - 300)]
    row_expert = torch.where(live, experts, -1)[at].numpy()
    if al is None:
        wc, ws = wc[0], ws[0]
    for silu in (False, True) if N % 32 == 0 else (False,):
        mark = torch.full((M, N // 2 if silu else N), -9.5, dtype=torch.bfloat16, device="cuda")
        y = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=al, silu_mul=silu, out=mark.clone())
        check_product(np64(y[at.cuda()]), torch.bfloat16, x64[at.numpy()], w64, row_expert, silu, K,
                      f"silu {silu}")
        assert bool((y[(~live & (experts >= 0)).cuda()] == 0).all())
        assert torch.equal(y[(experts < 0).cuda()], mark[(experts < 0).cuda()])


# ---------------------------------------------------------------------------
# rows: short ones, unaligned ones, more than one launch takes at once
# ---------------------------------------------------------------------------
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "u8": torch.uint8}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
INT_MIN = -(1 << 31)


def values(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    if dtype == torch.uint8:
        return torch.randint(0, 256, shape, generator=g, dtype=dtype).cuda()
    return torch.randn(*shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("u8", "u8")])
@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 7, 8, 9, 11, 15, 16, 17, 23, 31])
def test_short_rows(H, dtype, out):
    """Rows shorter than 16 bytes go element by element, longer ones in pieces of 16 whose
    last one overlaps; bounds as in test_gpu_rows."""
    T, k, E = 70, 3, 7
    ids = some_ids(T, k, E, 50)
    ids.view(-1)[::5] = -1
    al = binding.moe_lora_align(ids, no_slots(T), None, E, 0, 16, pair_rows=True)
    cap, used = al["capacity"], int(al["num_rows_padded"].cpu()[0])
    pr = ro.pair_rows_of(al["sorted_pair_ids"][:cap].cpu().numpy(), T * k)
    assert (pr < 0).any()
    x = values((T, H), DT[dtype], 51)
    mark = values((cap, H), DT[dtype], 52)
    got = binding.moe_lora_permute(x, al, k, out=mark.clone())
    ref = ro.permute(x.float().cpu().numpy(), pr, k, cap)[0]
    assert np.array_equal(got[:used].float().cpu().numpy(), ref[:used])
    assert torch.equal(got[used:], mark[used:])
    if dtype == "u8":
        return
    rows, dy = values((cap, H), DT[dtype], 53), values((T, H), DT[out], 55)
    w = values((T, k), torch.float32, 54)
    ho, hr = HALF[DT[out]], HALF[DT[dtype]]
    for weights_ in (w, None):
        y = binding.moe_lora_unpermute(rows, al, k, weights_, out_dtype=DT[out])
        ref, mag = ro.unpermute(np64(rows), pr, k, None if weights_ is None else np64(w))
        assert np.all(np.abs(np64(y) - ref) <= k * 2.0 ** -24 * mag * (1 + ho) + ho * np.abs(ref))
    d_rows, d_w = binding.moe_lora_unpermute_backward(dy, rows, al, k, w, d_rows=mark.clone())
    ref, ref_w, mag_w = ro.unpermute_backward(np64(dy), np64(rows), pr, k, np64(w), cap)
    assert np.all(np.abs(np64(d_rows) - ref)[:used] <= (2.0 ** -24 * (1 + hr) + hr) * np.abs(ref[:used]))
    assert torch.equal(d_rows[used:], mark[used:])
    assert np.all(np.abs(np64(d_w) - ref_w) <= (H + 1) * 2.0 ** -24 * mag_w)


@pytest.mark.parametrize("H", [3, 9, 264, 1001])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_unaligned_pointers_change_no_bit(H, dt):
    """Whatever its pointers are aligned to, a call takes the same pieces in the same order."""
    T, k, E = 23, 2, 4
    al = binding.moe_lora_align(some_ids(T, k, E, 60), no_slots(T), None, E, 0, 16, pair_rows=True)
    cap, used = al["capacity"], int(al["num_rows_padded"].cpu()[0])

    def odd(t, by):
        return torch.cat((t.new_zeros(by), t.reshape(-1)))[by:].view(t.shape)

    x, rows, w = values((T, H), dt, 61), values((cap, H), dt, 62), values((T, k), torch.float32, 63)
    want = (binding.moe_lora_permute(x, al, k)[:used], binding.moe_lora_unpermute(rows, al, k, w),
            binding.moe_lora_permute_backward(rows, al, k),
            *binding.moe_lora_unpermute_backward(x, rows, al, k, w))
    for by in (1, 3):
        xo, ro_, wo = odd(x, by), odd(rows, by), odd(w, by)
        got = (binding.moe_lora_permute(xo, al, k, out=odd(rows, by))[:used],
               binding.moe_lora_unpermute(ro_, al, k, wo, y=odd(x, by)),
               binding.moe_lora_permute_backward(ro_, al, k, dx=odd(x, by)),
               *binding.moe_lora_unpermute_backward(xo, ro_, al, k, wo, d_rows=odd(rows, by),
                                                    d_weights=odd(w, by)))
        for i, (a, b) in enumerate(zip(got, want)):
            n = used if i in (0, 3) else len(a)
            assert torch.equal(a[:n], b[:n]), (by, i)


def test_tokens_of_more_than_one_round():
    """More tokens than one launch has workgroups (2^22): every one of them, with some that
    have no row."""
    T, H = (1 << 22) + 1037, 5
    say("tokens of more than one round")
    g = torch.Generator(device="cuda").manual_seed(70)
    perm = torch.randperm(T, generator=g, device="cuda").int()
    gone = torch.arange(T, device="cuda") % 1000 == 3
    pr = torch.where(gone, -1, perm)
    ids = torch.full((T,), T, dtype=torch.int32, device="cuda")
    ids[perm[~gone].long()] = torch.arange(T, dtype=torch.int32, device="cuda")[~gone]
    al = dict(sorted_pair_ids=ids, pair_rows=pr, capacity=T,
              num_rows_padded=torch.tensor([T], dtype=torch.int32, device="cuda"))
    x = torch.randn(T, H, generator=g, device="cuda")
    w = torch.rand(T, 1, generator=g, device="cuda")
    want = torch.zeros(T, H, device="cuda")
    want[perm[~gone].long()] = x[~gone]
    rows = binding.moe_lora_permute(x, al, 1, out=torch.full_like(x, 9.0))
    assert torch.equal(rows, want)
    there = x * ~gone.view(-1, 1)
    assert torch.equal(binding.moe_lora_unpermute(rows, al, 1, w), there * w)     # one product each
    assert torch.equal(binding.moe_lora_permute_backward(rows, al, 1), there)
    d_rows, d_w = binding.moe_lora_unpermute_backward(x, rows, al, 1, w, d_rows=torch.full_like(x, 9.0))
    want[perm[~gone].long()] = (x * w)[~gone]
    assert torch.equal(d_rows, want)
    ref = (x.double() * there.double()).sum(1, keepdim=True)
    assert bool(((d_w.double() - ref).abs() <= (H + 1) * 2.0 ** -24 * ref).all())    # a sum of squares


def test_padding_of_more_than_one_round():
    """More rows than one launch's workgroups look at (2^20 x 16): padding among them and at
    the end gets zeros, rows behind num_rows_padded stay."""
    R, used = (1 << 24) + 5000, (1 << 24) + 4711
    say("padding of more than one round")
    ids = torch.full((R,), 3, dtype=torch.int32, device="cuda")
    at = torch.tensor([7, 1 << 23, (1 << 24) + 4600], device="cuda")
    ids[at] = torch.arange(3, dtype=torch.int32, device="cuda")
    al = dict(sorted_pair_ids=ids, pair_rows=at.int(), capacity=R,
              num_rows_padded=torch.tensor([used], dtype=torch.int32, device="cuda"))
    x = torch.tensor([[1.0], [2.0], [3.0]], device="cuda")
    want = torch.zeros(R, 1, device="cuda")
    want[at] = x
    want[used:] = 9.0
    assert torch.equal(binding.moe_lora_permute(x, al, 1, out=torch.full_like(want, 9.0)), want)
    d_rows, _ = binding.moe_lora_unpermute_backward(x, None, al, 1, d_rows=torch.full_like(want, 9.0))
    assert torch.equal(d_rows, want)


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("part", range(8))
def test_quantise_each_finite_bf16_value(part):
    """Every finite bf16 value as a block's largest, beside smaller ones of both signs."""
    v = (torch.arange(part, 0x7F80, 8, dtype=torch.int32) << 16).view(torch.float32)
    x = v.view(-1, 1) * torch.linspace(-1, 1, 32).view(1, -1)
    x[:, 0] = -v
    x = x.bfloat16()
    codes, scales = binding.moe_lora_mx4_quantize(x.cuda())
    rc, rs = ro.mx4_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)


def test_quantise_more_than_one_round():
    """More values than one launch takes at once (2^20 x 256 x 4 units of 8): every row as
    its pattern says, there and back."""
    rows, cols, period = (1 << 20) + 77, 8224, 16
    say("quantise more than one round")
    assert rows * cols > 1 << 33
    pattern = values((period, cols), torch.bfloat16, 80)
    x = pattern.repeat(-(-rows // period), 1)[:rows]
    codes, scales = binding.moe_lora_mx4_quantize(x)
    rc, rs = binding.moe_lora_mx4_quantize(pattern)
    assert np.array_equal(rc.cpu().numpy(), ro.mx4_quantize(np64(pattern))[0])
    for got, want in ((codes, rc), (scales, rs)):
        for r in range(0, rows, period << 10):
            part = got[r:r + (period << 10)]
            assert torch.equal(part, want.repeat(-(-len(part) // period), 1)[:len(part)]), r
    back = binding.moe_lora_mx4_dequantize(codes, scales)
    want = binding.moe_lora_mx4_dequantize(rc, rs)
    for r in range(0, rows, period << 10):
        part = back[r:r + (period << 10)]
        assert torch.equal(part, want.repeat(-(-len(part) // period), 1)[:len(part)]), r


# ---------------------------------------------------------------------------
# calls that the documentation allows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("bm,n,N", [(16, 9, 96), (32, 40, 1040), (64, 9, 96), (64, 40, 528), (128, 40, 528),
                                    (192, 24, 528), (256, 35, 2064)])
def test_tiles_of_other_experts(bm, n, N, kind):
    """Tiles of an expert that the weights do not hold, in the middle, at the start and at the
    end: their rows stay as they were, the others are theirs."""
    E, K = 3, 160
    say(f"tiles of other experts {kind} block_m {bm} x {n}")
    g = torch.Generator().manual_seed(90)
    tiles = torch.randint(-1, E + 2, (n,), generator=g)
    tiles[0], tiles[1], tiles[-1] = E, 1, INT_MIN
    al = dict(block_m=bm, tile_expert=tiles.int().cuda())
    wc, ws, w64 = weights(E, N, K, 91)
    x, xs, x64 = activations(n * bm, K, kind, 92)
    row_expert = torch.where((tiles >= 0) & (tiles < E), tiles, -1).numpy().repeat(bm)
    mark = torch.full((n * bm, N), -9.5, dtype=torch.float32, device="cuda")
    y = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=al, out=mark.clone())
    check_product(np64(y), torch.float32, x64, w64, row_expert, False, K, "other experts")
    other = torch.from_numpy(row_expert < 0).cuda()
    assert torch.equal(y[other], mark[other])


def test_an_expert_named_twice_by_a_token():
    """Both pairs have a row of their own, and both count."""
    T, k, E, H = 50, 4, 4, 96
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(93)).int().cuda()
    al = binding.moe_lora_align(ids, no_slots(T), None, E, 0, 16, pair_rows=True)
    x, w = values((T, H), torch.float32, 94), values((T, k), torch.float32, 95)
    pr = al["pair_rows"]
    assert len(set(pr.tolist())) == T * k and bool((pr >= 0).all())
    rows = binding.moe_lora_permute(x, al, k)
    assert torch.equal(rows[pr.long()].view(T, k, H), x.unsqueeze(1).expand(T, k, H))
    y = binding.moe_lora_unpermute(rows, al, k, w)
    ref = np64(x) * np64(w).sum(1, keepdims=True)
    mag = np.abs(np64(x)) * np.abs(np64(w)).sum(1, keepdims=True)
    assert np.all(np.abs(np64(y) - ref) <= (k + 1) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("activations_", ["bf16", "mx4"])
def test_layer_captured_and_on_two_streams(activations_):
    """run_mx4_layer replayed from a graph with new tokens, experts and weights, beside its own
    eager calls, and on two streams at once."""
    T, k, E, H, I = 150, 2, 6, 256, 96  # noqa: E741
    guc, gus, _ = weights(E, 2 * I, H, 96)
    dc, ds, _ = weights(E, H, I, 97)

    def batch(seed):
        return dict(x=values((T, H), torch.bfloat16, seed), topk_ids=some_ids(T, k, E, seed),
                    topk_weights=values((T, k), torch.float32, seed + 1))

    layer = dict(w_gate_up_mx4=(guc, gus), w_down_mx4=(dc, ds))
    now = dict(batch(100), **layer)
    binding.run_mx4_layer(now, activations_)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = binding.run_mx4_layer(now, activations_)
    for i in range(4):
        for name, t in batch(110 + i).items():
            now[name].copy_(t)
        want = binding.run_mx4_layer(now, activations_)
        torch.cuda.synchronize()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
    batches = [dict(batch(120 + i), **layer) for i in range(2)]
    want = [binding.run_mx4_layer(b, activations_) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(binding.run_mx4_layer(batches[i], activations_))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[i]) for i in range(2) for a in got[i])


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("bm,n", [(16, 3), (64, 3), (64, 5), (256, 3)])
def test_weights_past_4_gib(kind, bm, n):
    """The last experts of more than 4 GiB of codes and 256 MiB of scales: the bits of the same
    call on those weights alone."""
    E, N, K = 66, 8192, 16384
    say(f"weights past 4 GiB {kind} block_m {bm} x {n}")
    g = torch.Generator(device="cuda").manual_seed(130)
    wc = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(120, 126, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    assert wc.numel() > 1 << 32
    x, xs, _ = activations(n * bm, K, kind, 131)
    tiles = torch.tensor([E - 1, 0, E - 2] + [E - 1] * (n - 3), dtype=torch.int32, device="cuda")
    few = torch.tensor([0, E - 2, E - 1], device="cuda")
    alone = torch.tensor([2, 0, 1] + [2] * (n - 3), dtype=torch.int32, device="cuda")
    y, want = (binding.moe_lora_mx4_gemm(x, c, s, x_scales=xs, align_out=dict(block_m=bm, tile_expert=t))
               for c, s, t in ((wc, ws, tiles), (wc[few], ws[few], alone)))
    assert torch.equal(y, want) and bool(y.isfinite().all()) and float(y.abs().max()) > 0


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("bm", [16, 64, 256, None])
@pytest.mark.parametrize("what", ["out", "x"])
def test_rows_past_4_gib(kind, bm, what):
    """x or out of more than 4 GiB: rows from all over, against the oracle."""
    dt = torch.bfloat16
    M, N, K = (1 << 17, 16480, 32) if what == "out" else (1 << 18, 32, 9280 if kind == "bf16" else 33792)
    say(f"rows past 4 GiB {kind} block_m {bm} {M} x {N} x {K}")
    g = torch.Generator(device="cuda").manual_seed(132)
    if kind == "bf16":
        x, xs = torch.randn(M, K, generator=g, device="cuda").to(dt), None
    else:
        x = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        xs = torch.randint(120, 126, (M, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    assert (M * N * 2 if what == "out" else x.nbytes) > 1 << 32
    wc, ws, w64 = weights(1, N, K, 133)
    al = None
    if bm is None:
        wc, ws = wc[0], ws[0]
    else:
        al = dict(block_m=bm, tile_expert=torch.zeros(M // bm, dtype=torch.int32, device="cuda"))
    y = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=al)
    at = torch.cat((torch.arange(0, M, 1021), torch.arange(M - 70, M))).cuda()
    x64 = np64(x[at]) if xs is None else ro.mx4_values(x[at].cpu().numpy(), xs[at].cpu().numpy())
    check_product(np64(y[at]), dt, x64, w64, np.zeros(len(at), int), False, K, "rows")
