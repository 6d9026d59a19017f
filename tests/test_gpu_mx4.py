"""MX4 quantisation and products against the float64 oracle.

Codes, scales and dequantised values are exact.  A product sum of K fp32 terms
(each product of a bf16 or e2m1 value with an e2m1 value is exact) is off by at most
K * 2^-23 of the sum of the terms' magnitudes (one addition per term, each off by
at most one step whatever the matrix core's rounding); the output type adds half a
step."""
import numpy as np
import pytest
import torch

from oracle import rows_mx4_oracle as ro
from gpu_helpers import say
from moe_expert_layer_segment_amd import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def special_values():
    """Blocks with ties, borders of the scale, zeros, denormals, infinities, NaN."""
    rows = []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.0])
    for e in (-120, -3, 0, 5, 120):
        rows.append(np.concatenate((ties, -ties)) * 2.0 ** e)
    rows.append(np.zeros(32))
    rows.append(np.full(32, -0.0))
    tiny = np.zeros(32)
    tiny[3], tiny[7] = 2.0 ** -133, -(2.0 ** -126)       # bf16 denormal, smallest normal
    rows.append(tiny)
    only = np.zeros(32)
    only[5] = 2.0 ** -133
    rows.append(only)
    rows.append(np.linspace(-1, 1, 32) * 2.0 ** -128)
    big = np.linspace(-1, 1, 32) * 3.3e38                 # near the largest finite bf16
    rows.append(big)
    edge = np.full(32, 1.0)
    edge[0] = 4.0 - 2.0 ** -6                             # just below the next scale
    rows.append(edge)
    edge = edge.copy()
    edge[0] = 4.0
    rows.append(edge)
    for bad in (np.inf, -np.inf, np.nan):
        b = np.linspace(-3, 3, 32)
        b[17] = bad
        rows.append(b)
    return np.concatenate(rows).reshape(1, -1)


def check_quantize(x):
    codes, scales = binding.moe_lora_mx4_quantize(x)
    torch.cuda.synchronize()
    rc, rs = ro.mx4_quantize(np64(x))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    ref = ro.mx4_values(rc, rs)
    for dt in (torch.float32, torch.bfloat16):
        got = np64(binding.moe_lora_mx4_dequantize(codes, scales, out_dtype=dt))
        with np.errstate(over="ignore"):
            assert np.array_equal(got, ref.astype(np.float32).astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_special_values(dtype):
    check_quantize(torch.from_numpy(special_values()).to(DT[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (5, 7, 160), (64, 2048), (2, 32 * 131)])
def test_quantize_shapes(shape, dtype):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-40, 40, (*shape[:-1], 1), generator=g))
    check_quantize(x.to(DT[dtype]).cuda())


def test_quantize_every_bf16_value():
    """Every finite bf16 value as the block's largest, beside smaller ones."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    v = (bits << 16).view(torch.float32)
    x = v.view(-1, 1) * torch.linspace(-1, 1, 32).view(1, -1)
    x[:, 0] = -v
    check_quantize(x[::7].bfloat16().cuda())


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).view(16, 16).repeat(16, 1)     # [256, 16]
    codes = codes.view(16, 16, 16).repeat(16, 1, 1).view(-1, 16)               # each under every scale
    scales = torch.arange(256, dtype=torch.uint8).view(-1, 1).repeat(1, 16).view(-1, 1)
    ref = ro.mx4_values(codes.numpy(), scales.numpy())
    for dt in (torch.float32, torch.bfloat16):
        got = np64(binding.moe_lora_mx4_dequantize(codes.cuda(), scales.cuda(), out_dtype=dt))
        with np.errstate(over="ignore"):
            assert np.array_equal(got, ref.astype(np.float32).astype(np.float64), equal_nan=True)


def test_quantize_rows_used():
    """Rows from the device count on keep what their outputs held."""
    x = torch.randn(40, 96, device="cuda").bfloat16()
    codes, scales = binding.moe_lora_mx4_quantize(x)
    for used in (0, 1, 17, 40, 99):
        c = torch.full_like(codes, 0xCD)
        s = torch.full_like(scales, 0xCD)
        binding.moe_lora_mx4_quantize(x, torch.tensor([used], dtype=torch.int32, device="cuda"), c, s)
        n = min(used, 40)
        assert torch.equal(c[:n], codes[:n]) and torch.equal(s[:n], scales[:n])
        assert bool((c[n:] == 0xCD).all()) and bool((s[n:] == 0xCD).all())


def weights(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(E, N, K, generator=g) * K ** -0.5 * torch.exp2(torch.randint(-2, 3, (E, N, 1), generator=g))
    codes, scales = binding.moe_lora_mx4_quantize(w.cuda())
    return codes, scales, ro.mx4_values(codes.cpu().numpy(), scales.cpu().numpy())


def activations(M, K, kind, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    if kind == "bf16":
        return x, None, np64(x)
    codes, scales = binding.moe_lora_mx4_quantize(x)
    return codes, scales, ro.mx4_values(codes.cpu().numpy(), scales.cpu().numpy())


def check_product(got, out_dtype, x64, w64, row_expert, silu, K, what):
    half = HALF[out_dtype]
    err = K * 2.0 ** -23
    if not silu:
        ref, mag = ro.mx4_gemm(x64, w64, row_expert)
        bound = err * mag * (1 + half) + half * np.abs(ref)
    else:
        ref, (g, u, s, mg, mu) = ro.mx4_gemm(x64, w64, row_expert, True)
        # |silu'| <= 1.1; SiLU itself: exp2 of an argument off by |g| * 2^-23, a
        # reciprocal and two products of a few steps each
        bound = (1.1 * np.abs(u) + err * mu) * err * mg + np.abs(s) * err * mu \
            + np.abs(ref) * (np.abs(g) + 8) * 2.0 ** -23
        bound = bound * (1 + half) + half * np.abs(ref) + 2.0 ** -126
    live = np.asarray(row_expert) >= 0
    off = np.abs(got - ref)[live]
    assert np.all(np.isfinite(got[live])), what
    worst = float(np.max(off / np.maximum(bound[live], 1e-300))) if off.size else 0.0
    rel = float(np.linalg.norm(off) / max(np.linalg.norm(ref[live]), 1e-30)) if off.size else 0.0
    say(f"  {what}: rel {rel:.2e}, {worst:.3f} of the bound")
    assert worst <= 1.0, what


DENSE = [(1, 16, 32), (1, 2112, 736), (5, 48, 96), (16, 64, 256), (17, 80, 288), (33, 32, 512),
         (64, 128, 1056), (100, 272, 480), (129, 256, 256), (300, 96, 2080), (513, 528, 1312),
         (257, 1040, 768),
         # past 64 tiles of 64 x 256
         (64, 16640, 736), (70, 16400, 288), (130, 8208, 544), (520, 2064, 1312), (1100, 1040, 2080),
         (700, 1536, 2560), (1000, 1056, 1568), (4129, 288, 96)]


@pytest.mark.parametrize("shape", DENSE, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind", ["bf16", "mx4"])
def test_dense_product(shape, kind):
    M, N, K = shape
    say(f"dense product {shape} {kind}")
    wc, ws, w64 = weights(1, N, K, 2)
    x, xs, x64 = activations(M, K, kind, 3)
    for dt in (torch.float32, torch.bfloat16):
        y = binding.moe_lora_mx4_gemm(x, wc[0], ws[0], x_scales=xs, out_dtype=dt)
        check_product(np64(y), dt, x64, w64, np.zeros(M, int), False, K, f"{dt}")
    if N % 32 == 0:
        y = binding.moe_lora_mx4_gemm(x, wc[0], ws[0], x_scales=xs, silu_mul=True)
        check_product(np64(y), torch.bfloat16, x64, w64, np.zeros(M, int), True, K, "silu_mul")


GROUPED = [  # experts of the tiles (-1: unused), block_m, N, K
    ([0, 0, 2, 1, -1, -1], 16, 64, 256),
    ([3, 3, 1, -1], 32, 96, 160),
    ([0, 2, 2, -1], 48, 112, 320),
    ([1, 0, 2], 64, 160, 544),
    ([1, 0, -1, -1], 128, 288, 512),
    ([2, 0, 1], 256, 544, 800),
    ([2, 2, 1, 1, 0, -1], 256, 256, 2304),
    ([-1, -1], 128, 64, 64),
    ([0, 0, 2, 1, 3] * 8 + [-1], 64, 544, 800),
    ([1, 1, 3, 0, 2] * 4 + [-1], 128, 544, 2304),
    ([3, 2, 2, 0, 1, 3, 0], 256, 800, 1056),
    ([1, 0, 0, -1], 48, 64, 256),
    ([2, 0, 1, -1], 96, 112, 320),
    ([2, 0, 1, 3] * 6 + [-1], 192, 528, 544),
]


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: f"b{c[1]}N{c[2]}K{c[3]}")
@pytest.mark.parametrize("kind", ["bf16", "mx4"])
def test_grouped_product(case, kind):
    tiles, bm, N, K = case
    say(f"grouped product {case} {kind}")
    E, M = 4, len(tiles) * bm
    wc, ws, w64 = weights(E, N, K, 4)
    x, xs, x64 = activations(M, K, kind, 5)
    al = dict(block_m=bm, tile_expert=torch.tensor(tiles, dtype=torch.int32, device="cuda"))
    row_expert = np.repeat(tiles, bm)
    for silu in (False, True) if N % 32 == 0 else (False,):
        for dt in (torch.bfloat16, torch.float32):
            mark = torch.full((M, N // 2 if silu else N), -9.5, dtype=dt, device="cuda")
            y = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=al, silu_mul=silu,
                                          out=mark.clone())
            check_product(np64(y), dt, x64, w64, row_expert, silu, K, f"{dt} silu {silu}")
            unused = torch.from_numpy(row_expert < 0).cuda()
            assert torch.equal(y[unused], mark[unused]), "rows of unused tiles were written"


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("bm,times", [(16, 1), (256, 1), (64, 23), (256, 6)])
def test_rows_do_not_reach_other_rows(kind, bm, times):
    """NaN rows (what padding may hold) change no other row, bit for bit; a NaN scale of a
    weight row changes that output column alone."""
    E, N, K, tiles = 2, 96, 416, [1, 0, 1] * times
    M = bm * len(tiles)
    wc, ws, _ = weights(E, N, K, 6)
    al = dict(block_m=bm, tile_expert=torch.tensor(tiles, dtype=torch.int32, device="cuda"))
    x, xs, _ = activations(M, K, kind, 7)
    clean = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=al)
    bad = torch.arange(3, M, 5, device="cuda")
    x2, xs2 = x.clone(), None if xs is None else xs.clone()
    if kind == "bf16":
        x2[bad] = float("nan")
    else:
        xs2[bad] = 255
    y = binding.moe_lora_mx4_gemm(x2, wc, ws, x_scales=xs2, align_out=al)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[bad]).all())
    ws2 = ws.clone()
    ws2[1, 7, K // 32 - 1] = 255
    y = binding.moe_lora_mx4_gemm(x, wc, ws2, x_scales=xs, align_out=al)
    of1 = torch.tensor(tiles, device="cuda").repeat_interleave(bm) == 1
    assert bool(torch.isnan(y[of1, 7]).all())
    y[of1, 7] = clean[of1, 7]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("bm", [16, 32, 64, 128, 256])
def test_padding_rows_are_not_read(kind, bm):
    """With pair_rows in the layout the padding rows (NaN here) give zeros, the other
    rows the same bits as without it, and rows behind the last tile are untouched."""
    T, k, E, N, K = 90, 2, 5, 160, 544
    say(f"padding rows {kind} block_m {bm}")
    g = torch.Generator().manual_seed(15)
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).int().cuda()
    al = binding.moe_lora_align(ids, torch.full((T,), -1, dtype=torch.int32, device="cuda"), None, E, 0,
                                bm, pair_rows=True)
    used, M = int(al["num_rows_padded"].cpu()[0]), al["capacity"]
    assert used < M
    sid = al["sorted_pair_ids"]
    pad = (sid >= T * k).clone()
    wc, ws, w64 = weights(E, N, K, 16)
    x, xs, x64 = activations(M, K, kind, 17)
    (x if kind == "bf16" else xs)[pad] = torch.tensor(float("nan")).bfloat16() if kind == "bf16" else 255
    plain = {n: al[n] for n in ("block_m", "tile_expert")}
    row_expert = al["tile_expert"].cpu().numpy().repeat(bm)[:M]
    row_expert = np.where(pad.cpu().numpy(), -1, row_expert)
    for silu in (False, True):
        mark = torch.full((M, N // 2 if silu else N), -9.5, dtype=torch.float32, device="cuda")
        y = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=al, silu_mul=silu, out=mark.clone())
        check_product(np64(y), torch.float32, x64, w64, row_expert, silu, K, f"silu {silu}")
        assert bool((y[:used][pad[:used]] == 0).all())
        assert torch.equal(y[used:], mark[used:])
        z = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=plain, silu_mul=silu, out=mark.clone())
        assert torch.equal(y[~pad], z[~pad])


MANY = [  # block_m, tiles in use and behind them, N: past 256 workgroups, whose last round is split
    (256, 18, 2, 4096), (256, 21, 0, 4096), (256, 25, 1, 4096), (256, 31, 1, 2064), (128, 20, 3, 4096),
    (256, 36, 1, 1040), (128, 1, 0, 16), (256, 2, 1, 528), (64, 30, 2, 1040), (64, 70, 1, 272), (192, 24, 2, 1040), (192, 3, 1, 96)]


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"b{c[0]}t{c[1]}N{c[3]}")
@pytest.mark.parametrize("kind", ["bf16", "mx4"])
def test_many_tiles(case, kind):
    """Row tiles with any number of rows in use, with gaps; the others give zeros."""
    bm, tiles, behind, N = case
    E, K, M = 3, 96, bm * (tiles + behind)
    say(f"many tiles {case} {kind}")
    g = torch.Generator().manual_seed(18)
    experts = torch.cat((torch.randint(0, E, (tiles,), generator=g), torch.full((behind,), -1)))
    fill = torch.randint(0, bm + 1, (tiles + behind,), generator=g)
    for i, n in enumerate((0, 1, 64, 65, 128, bm)[:tiles]):
        fill[i] = n
    live = torch.arange(bm).view(1, -1) < fill.view(-1, 1)
    live &= torch.rand(tiles + behind, bm, generator=g) < 0.9
    live = live.reshape(-1)
    pairs = int(live.sum()) + 1
    sid = torch.full((M,), pairs, dtype=torch.int32)
    sid[live] = torch.randperm(pairs - 1, generator=g).int()
    sid[~live] = torch.where(torch.rand(int((~live).sum()), generator=g) < 0.5, -1, pairs).int()
    al = dict(block_m=bm, tile_expert=experts.int().cuda(), sorted_pair_ids=sid.cuda(),
              pair_rows=torch.empty(pairs, dtype=torch.int32, device="cuda"))
    wc, ws, w64 = weights(E, N, K, 19)
    x, xs, x64 = activations(M, K, kind, 20)
    row_expert = np.where(live.numpy(), experts.numpy().repeat(bm), -1)
    for silu in (False, True) if N % 32 == 0 else (False,):
        mark = torch.full((M, N // 2 if silu else N), -9.5, dtype=torch.bfloat16, device="cuda")
        y = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, align_out=al, silu_mul=silu, out=mark.clone())
        check_product(np64(y), torch.bfloat16, x64, w64, row_expert, silu, K, f"silu {silu}")
        used = bm * tiles
        assert bool((y[:used][~live[:used].cuda()] == 0).all())
        assert torch.equal(y[used:], mark[used:])


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("M", [1, 40, 300, 4200])
def test_extreme_scales(kind, M):
    """Scales at both ends of the e8m0 range; sums stay in fp32's."""
    N, K = 64, 128
    g = torch.Generator().manual_seed(8)
    wc = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    for wb, xb in ((0, 250), (1, 253), (253, 1), (127, 127), (200, 60)):
        ws = torch.full((N, K // 32), wb, dtype=torch.uint8, device="cuda")
        w64 = ro.mx4_values(wc.cpu().numpy(), ws.cpu().numpy())
        if kind == "mx4":
            x = torch.randint(0, 256, (M, K // 2), generator=g, dtype=torch.uint8).cuda()
            xs = torch.full((M, K // 32), xb, dtype=torch.uint8, device="cuda")
            x64 = ro.mx4_values(x.cpu().numpy(), xs.cpu().numpy())
        else:
            x = (torch.randint(-8, 9, (M, K), generator=g).double() * 2.0 ** (xb - 127)).bfloat16().cuda()
            xs, x64 = None, np64(x)
            # bf16 weights: 4 and 6 times 2^126 pass the largest finite value, 2^128 - 2^120
            w64 = np.where(np.abs(w64) >= 2.0 ** 128, np.copysign(np.inf, w64), w64)
        y = binding.moe_lora_mx4_gemm(x, wc, ws, x_scales=xs, out_dtype=torch.float32)
        if not (np.all(np.isfinite(x64)) and np.all(np.isfinite(w64))):
            # infinite values on one side (in bf16 also x of 2 * 2^126 and more): the sums are
            # infinite, or NaN
            with np.errstate(invalid="ignore"):
                ref = ro.mx4_gemm(x64, w64[None], np.zeros(M, int))[0]
            assert np.array_equal(np64(y), ref, equal_nan=True)
            continue
        check_product(np64(y), torch.float32, x64, w64[None], np.zeros(M, int), False, K,
                      f"scales {wb} {xb}")


def test_streams_and_graph():
    """Quantise, product, dequantise on a side stream and captured; replays equal the
    eager results with eager calls and new inputs between them."""
    M, N, K = 48, 128, 256
    wc, ws, _ = weights(1, N, K, 9)
    wc, ws = wc[0], ws[0]
    x = torch.randn(M, K, device="cuda").bfloat16()
    codes = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(M, K // 32, dtype=torch.uint8, device="cuda")
    y, z = (torch.empty(M, N, device="cuda") for _ in range(2))
    back = torch.empty_like(x)

    def step():
        binding.moe_lora_mx4_quantize(x, codes=codes, scales=scales)
        binding.moe_lora_mx4_gemm(codes, wc, ws, x_scales=scales, out=y)
        binding.moe_lora_mx4_gemm(x, wc, ws, out=z)
        binding.moe_lora_mx4_dequantize(codes, scales, out=back)
        return [t.clone() for t in (codes, scales, y, z, back)]

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
        x.copy_(torch.randn(M, K, device="cuda"))
        want = step()
        for t in (codes, scales, y, z, back):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (codes, scales, y, z, back))), i


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 64, 32), (27, 2, 8, 256, 96), (600, 3, 6, 320, 128),
                                       (2100, 2, 4, 128, 64)])
def test_layer_from_the_operators(kind, T, k, E, H, I):
    """run_mx4_layer against the layer's formula in float64 on the decoded weights.

    bf16 x: the activations between the products round to bf16 (2^-8 each), so y is
    off by at most 2^-8 of sum_j w |act| |W_down| plus fp32 sums.  MX4 x: the layer's
    own quantised activations are not determined to the last bit, so act is compared
    after each step through the operators instead, and y on them."""
    say(f"layer T{T} k{k} E{E} H{H} I{I} {kind}")
    g = torch.Generator().manual_seed(10)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    w = torch.rand(T, k, generator=g).cuda()
    w = w / w.sum(1, keepdim=True)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    guc, gus, gu64 = weights(E, 2 * I, H, 11)
    dc, ds, d64 = weights(E, H, I, 12)
    inputs = dict(x=x, topk_ids=ids, topk_weights=w, w_gate_up_mx4=(guc, gus), w_down_mx4=(dc, ds))
    y = np64(binding.run_mx4_layer(inputs, kind, out_dtype=torch.float32))
    if kind == "mx4":
        c, s = binding.moe_lora_mx4_quantize(x)
        x64 = ro.mx4_values(c.cpu().numpy(), s.cpu().numpy())
    else:
        x64 = np64(x)
    idn, wn = ids.cpu().numpy(), np64(w)
    ref, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = idn[t, j]
            gu = gu64[e] @ x64[t]
            act = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            if kind == "mx4":
                # bf16 rounding, then at most a quarter of the block's largest value
                # (half a step of 2 at 4..8 steps, or saturation from below 8 to 6)
                top = np.abs(act).reshape(-1, 32).max(1).repeat(32) * (1 + 2.0 ** -7)
                slack = 2.0 ** -7 * np.abs(act) + top / 4
            else:
                slack = 2.0 ** -7 * np.abs(act)
            ref[t] += wn[t, j] * (d64[e] @ act)
            bound[t] += wn[t, j] * (np.abs(d64[e]) @ (slack + 1e-5))
    worst = float(np.max(np.abs(y - ref) / bound))
    say(f"  {worst:.3f} of the bound")
    assert worst <= 1.0
    # step by step, from the layer's own calls
    bm = binding.mx4_block_m(T, k, E)
    al = binding.moe_lora_align(ids, torch.full((T,), -1, dtype=torch.int32, device="cuda"), None, E,
                                0, bm, pair_rows=True)
    used = int(al["num_rows_padded"].cpu()[0])
    if kind == "mx4":
        pc, ps = (binding.moe_lora_permute(t, al, k) for t in binding.moe_lora_mx4_quantize(x))
        act = binding.moe_lora_mx4_gemm(pc, guc, gus, x_scales=ps, align_out=al, silu_mul=True)
        ac, as_ = binding.moe_lora_mx4_quantize(act, al["num_rows_padded"])
        a64 = ro.mx4_values(ac[:used].cpu().numpy(), as_[:used].cpu().numpy())
        z = binding.moe_lora_mx4_gemm(ac, dc, ds, x_scales=as_, align_out=al, out_dtype=torch.float32)
    else:
        act = binding.moe_lora_mx4_gemm(binding.moe_lora_permute(x, al, k), guc, gus, align_out=al,
                                        silu_mul=True)
        a64 = np64(act[:used])
        z = binding.moe_lora_mx4_gemm(act, dc, ds, align_out=al, out_dtype=torch.float32)
    row_expert = al["tile_expert"][:used // bm].cpu().numpy().repeat(bm)
    check_product(np64(z[:used]), torch.float32, a64, d64, row_expert, False, I, "down")
    pr = al["pair_rows"].cpu().numpy()
    yr, mag = ro.unpermute(np64(z), pr, k, wn)
    assert np.all(np.abs(y - yr) <= (k + 1) * 2.0 ** -24 * mag)
