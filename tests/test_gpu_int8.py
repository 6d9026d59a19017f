"""8-bit integer rows, the norm in front of them and integer products against the float64
oracle.

Codes and scales of a quantisation are exact.  Those of the norm are held to the formula in 64
bits: a scale is one rounding to fp32 of a value that 64 bits leave 1e-14 off, so at most one
step away, and codes are those of the quotients by it but within 1e-9 of a border.  A product
before SiLU is exact to the bit: an integer rounded to fp32, times two scales.  SiLU(g) u adds
to the output type's half step: the exponential and the reciprocal a step (2^-23) each, the
correction of the exponent, the sum 1 + e and two products half a step each: 4 * 2^-23."""
import numpy as np
import pytest
import torch

from oracle import int8_balance_oracle as ib
from gpu_helpers import say
from moe_expert_layer_segment_amd import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -126          # below it fp32 (and bf16) have fewer digits


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rand(shape, dtype, seed, spread=8):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if x.dim() > 1:
        x = x * torch.exp2(torch.randint(-spread, spread + 1, (*shape[:-1], 1), generator=g).float())
    return x.to(DT[dtype]).cuda()


# ---------------------------------------------------------------------------
# quantize, dequantize
# ---------------------------------------------------------------------------
def check_quantize(x, codes, scales):
    rc, rs = ib.int8_quantize(np64(x))
    assert np.array_equal(scales.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), rc)
    for dt in (torch.float32, torch.bfloat16):
        got = binding.moe_lora_int8_dequantize(codes, scales, out_dtype=dt)
        assert got.dtype == dt and got.shape == codes.shape
        ref = (codes.float() * scales.unsqueeze(-1)).to(dt)
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.nan_to_num(), ref.nan_to_num())


def special_rows(n):
    """Rows with ties, zeros, denormals, infinities and NaN."""
    rows = []
    for e in (-120, -3, 0, 9, 118):                       # scale 2^e: every half is a tie
        v = (np.arange(n) % 255 - 127) + 0.5 * (np.arange(n) % 2)
        v[0] = 127
        rows.append(v.clip(-127, 127) * 2.0 ** e)
    rows.append(np.zeros(n))
    rows.append(np.full(n, -0.0))
    rows.append(np.full(n, 2.0 ** -133))                  # denormal in fp32 and bf16
    rows.append(np.linspace(-1, 1, n) * 2.0 ** -126)
    rows.append(np.linspace(-1, 1, n) * 3.3e38)
    for bad in (np.inf, -np.inf, np.nan):
        v = np.linspace(-3, 3, n)
        v[n // 2] = bad
        rows.append(v)
    return np.stack(rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 255, 1024, 40000])
def test_quantize_special_rows(n, dtype):
    x = torch.from_numpy(special_rows(n)).to(DT[dtype]).cuda()
    if dtype == "f32":
        extra = torch.full((1, n), 2.0 ** -149, device="cuda")   # its scale is 0
        x = torch.cat((x, extra))
    check_quantize(x, *binding.moe_lora_int8_quantize(x))


def test_quantize_next_to_borders():
    """fp32 values a step to either side of every border of two codes, under awkward scales."""
    for top in (1.0, 0.7312345, 3.3e-5, 12345.678):
        top = np.float32(top)
        scale = np.float32(np.float64(top) / 127)
        border = ((np.arange(-127, 127) + 0.5) * np.float64(scale)).astype(np.float32)
        row = np.concatenate([[top], border, np.nextafter(border, np.float32(np.inf), dtype=np.float32),
                              np.nextafter(border, np.float32(-np.inf), dtype=np.float32)])
        x = torch.from_numpy(row.reshape(1, -1)).cuda()
        check_quantize(x, *binding.moe_lora_int8_quantize(x))


# every number of pieces a thread takes, rows that 16 bytes do not divide, rows read twice
SHAPES = [(1, 1), (5, 7), (3, 8), (9, 64), (1, 257), (130, 511), (2, 3, 1000), (17, 1024), (7, 2049),
          (3, 4100), (2, 8200), (5, 16384), (2, 32768), (3, 32776), (2, 70001), (2100, 33), (9000, 40)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_shapes(shape, dtype):
    x = rand(shape, dtype, 1, 30)
    check_quantize(x, *binding.moe_lora_int8_quantize(x))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [40, 333, 5000, 40000])
def test_quantize_rows_used(cols, dtype):
    """Rows behind num_rows_used, and what lies behind odd rows, stay as they were."""
    x = rand((37, cols), dtype, 2)
    for used in (0, 1, 20, 37, 50, -3):
        codes = torch.full((37, cols), 99, dtype=torch.int8, device="cuda")
        scales = torch.full((37,), -5.0, device="cuda")
        n = torch.tensor([used], dtype=torch.int32, device="cuda")
        got = binding.moe_lora_int8_quantize(x, n, codes, scales)
        assert got[0] is codes and got[1] is scales
        at = max(0, min(used, 37))
        rc, rs = ib.int8_quantize(np64(x[:at]))
        assert np.array_equal(codes[:at].cpu().numpy(), rc) and np.array_equal(scales[:at].cpu().numpy(), rs)
        assert bool((codes[at:] == 99).all()) and bool((scales[at:] == -5).all())


def test_no_rows():
    c, s = binding.moe_lora_int8_quantize(torch.empty(0, 5, device="cuda"))
    assert c.shape == (0, 5) and s.shape == (0,)
    assert binding.moe_lora_int8_dequantize(c, s).shape == (0, 5)
    w = torch.ones(5, device="cuda")
    c, s, h, y = binding.moe_lora_rms_norm_quantize(torch.empty(0, 5, device="cuda"), w)
    assert c.shape == (0, 5) and h is None and y is None


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def check_norm(x, w, eps, res, codes, scales, h_out, y):
    h, n = ib.rms_norm(np64(x), np64(w), eps, None if res is None else np64(res))
    rs = ib.int8_scales(n).astype(np.float64)
    gs = scales.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(gs), np.isnan(rs))
    fine = ~np.isnan(rs)
    assert (np.abs(gs - rs)[fine] <= 2.0 ** -23 * rs[fine] + 2.0 ** -149).all()
    q = ib.int8_quotients(n, gs)
    got = codes.cpu().numpy().astype(np.float64)
    border = np.abs(np.abs(q - np.floor(q)) - 0.5) < 1e-9
    assert (border[fine] & (np.abs(q[fine]) < 126.9)).mean() < 0.01 or n.size < 1000
    ref = np.clip(np.rint(q), -127, 127)
    assert np.array_equal(np.where(border, 0, got), np.where(border, 0, ref))
    assert (np.abs(got - q)[fine] <= 0.5 + 1e-5).all()
    for out, exact in ((h_out, h), (y, n)):
        if out is None:
            continue
        got = np64(out)
        with np.errstate(invalid="ignore", over="ignore"):
            top = np.isnan(exact) | (np.abs(exact) >= 3.3e38)
            tol = HALF[out.dtype] * (1 + 2.0 ** -14) * np.abs(exact) + 2.0 ** -133
            assert (np.abs(got - exact)[~top] <= tol[~top]).all()
            assert np.array_equal(np.isnan(got[top]), np.isnan(exact[top]))


NORM_SHAPES = [(1, 1), (4, 3), (3, 8), (2, 5, 64), (7, 511), (5, 1000), (33, 1024), (6, 2050), (3, 4099),
               (130, 7168), (2, 8193), (3, 16384), (2500, 24)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm(shape, dtype):
    say(f"norm {shape} {dtype}")
    x, res = rand(shape, dtype, 3), rand(shape, dtype, 4)
    for wdt in ("f32", "bf16"):
        w = (1 + 0.3 * rand((shape[-1],), "f32", 5)).to(DT[wdt])
        for r in (None, res):
            for ydt in (None, torch.float32, torch.bfloat16):
                out = binding.moe_lora_rms_norm_quantize(x, w, 1e-5, residual=r, y_dtype=ydt)
                assert (out[2] is None) == (r is None) and (out[3] is None) == (ydt is None)
                check_norm(x, w, 1e-5, r, *out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [3, 40, 1031, 7168, 16383])
def test_norm_in_place(H, dtype):
    """residual_out may be the residual, or x; the results are the same bits."""
    x, res, w = rand((19, H), dtype, 6), rand((19, H), dtype, 7), rand((H,), dtype, 8)
    ref = binding.moe_lora_rms_norm_quantize(x, w, 1e-6, residual=res, y_dtype=torch.float32)
    for which in (0, 1):
        a, b = x.clone(), res.clone()
        out = binding.moe_lora_rms_norm_quantize(a, w, 1e-6, residual=b, residual_out=(b, a)[which],
                                                 y_dtype=torch.float32)
        assert out[2] is (b, a)[which]
        assert all(torch.equal(p, q) for p, q in zip(out, ref))


@pytest.mark.parametrize("H", [5, 64, 3000, 12000])
def test_norm_special_rows(H):
    """Zeros, values whose squares pass fp32's range, infinities, NaN, a weight of NaN."""
    x = torch.randn(9, H, generator=torch.Generator().manual_seed(9)).cuda()
    w = 1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(10)).cuda()
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, H // 2] = float("inf")
    x[4, 0] = float("nan")
    x[5] = 0
    x[5, H - 1] = -3
    x[6] = torch.finfo(torch.float32).min
    x[7] = 2.0 ** -140
    for eps in (1e-6, 0.0):
        check_norm(x, w, eps, None, *binding.moe_lora_rms_norm_quantize(x, w, eps, y_dtype=torch.float32))
    w[H - 1] = float("nan")
    codes, scales, _, y = binding.moe_lora_rms_norm_quantize(x, w, 1e-6, y_dtype=torch.float32)
    assert bool(scales.isnan().all()) and not bool(codes.any())
    assert bool(y[:, H - 1].isnan().all()) and not bool(y[0, :H - 1].any())


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def int8_weights(E, N, K, seed):
    """(codes [E, N, K], scales [E, N]) with every code there is, -128 too."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-128, 128, (E, N, K), generator=g, dtype=torch.int8)
    scales = torch.exp2(torch.randint(-14, -6, (E, N), generator=g).float()) * (1 + torch.rand(E, N, generator=g))
    return codes.cuda(), scales.cuda()


def int8_rows(M, K, seed):
    c, s = int8_weights(1, M, K, seed)
    return c[0], s[0]


def silu64(y):
    n = y.shape[1] // 2
    g, u = y[:, :n].astype(np.float64), y[:, n:].astype(np.float64)
    return g / (1 + np.exp(-g)) * u, np.abs(u)


def check_product(out, x, xs, w, ws, row_expert, silu):
    """Rows with a negative expert are not looked at."""
    y = ib.int8_product(x.cpu().numpy(), xs.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy(), row_expert)
    rows = slice(None) if row_expert is None else row_expert >= 0
    if not silu:
        ref = torch.from_numpy(y).to(out.dtype)
        assert torch.equal(out.cpu()[rows], ref[rows])
        return
    with np.errstate(over="ignore"):
        ref, up = silu64(y)
    tol = (4 * 2.0 ** -23 + HALF[out.dtype]) * np.abs(ref) + 128 * TINY * (up + 1)
    bad = np.abs(np64(out) - ref)[rows] > tol[rows]
    assert not bad.any(), (int(bad.sum()), bad.size)


def product(x, xs, w, ws, al=None, silu=False, dt=torch.bfloat16, mark=None, top_k=None):
    return binding.moe_lora_int8_gemm(x, xs, w, ws, align_out=al, silu_mul=silu, out=mark, out_dtype=dt,
                                      top_k=top_k)


DENSE = [(1, 16, 16), (1, 2112, 7168), (2, 32, 64), (17, 96, 48), (33, 64, 1040), (40, 288, 4112), (64, 512, 528),
         (100, 4112, 272), (129, 800, 656), (300, 1040, 416), (700, 528, 2064), (1000, 256, 96), (1500, 4096, 128),
         (4200, 272, 144)]


@pytest.mark.parametrize("shape", DENSE, ids=str)
def test_dense_product(shape):
    M, N, K = shape
    say(f"dense product {shape}")
    w, ws = int8_weights(1, N, K, 11)
    x, xs = int8_rows(M, K, 12)
    for silu in (False, True) if N % 32 == 0 else (False,):
        for dt in (torch.bfloat16, torch.float32):
            out = product(x, xs, w[0], ws[0], silu=silu, dt=dt)
            check_product(out, x, xs, w[0], ws[0], None, silu)


GROUPED = [  # tiles' experts, block_m, N, K
    ([0, 2, 2, 1, -1], 16, 96, 272), ([1, 0, 3], 32, 528, 144), ([3, -1, 0, 0, 1, -1], 16, 64, 4112),
    ([1, 0, 2], 64, 160, 544), ([1, 0, -1, -1], 128, 288, 512), ([2, 0, 1], 256, 544, 800),
    ([2, 2, 1, 1, 0, -1], 256, 256, 2304), ([-1, -1], 128, 64, 64), ([0, 0, 2, 1, 3] * 8 + [-1], 64, 544, 800),
    ([1, 1, 3, 0, 2] * 4 + [-1], 128, 544, 2304), ([3, 2, 2, 0, 1, 3, 0], 256, 800, 1056),
    ([1, 0, 0, -1], 48, 64, 256), ([2, 0, 1, -1], 96, 112, 320), ([2, 0, 1, 3] * 6 + [-1], 192, 528, 544)]


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: f"b{c[1]}N{c[2]}K{c[3]}")
def test_grouped_product(case):
    tiles, bm, N, K = case
    say(f"grouped product {case}")
    E, M = 4, len(tiles) * bm
    w, ws = int8_weights(E, N, K, 13)
    x, xs = int8_rows(M, K, 14)
    al = dict(block_m=bm, tile_expert=torch.tensor(tiles, dtype=torch.int32, device="cuda"))
    row_expert = np.repeat(tiles, bm)
    unused = torch.from_numpy(row_expert < 0).cuda()
    for silu in (False, True) if N % 32 == 0 else (False,):
        for dt in (torch.bfloat16, torch.float32):
            mark = torch.full((M, N // 2 if silu else N), -9.5, dtype=dt, device="cuda")
            y = product(x, xs, w, ws, al, silu, dt, mark.clone())
            check_product(y, x, xs, w, ws, row_expert, silu)
            assert torch.equal(y[unused], mark[unused]), "rows of unused tiles were written"


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("bm,T", [(16, 90), (32, 90), (64, 90), (64, 2100), (128, 90), (256, 90), (256, 3000), (192, 700)])
def test_padding_rows(bm, T, gather):
    """Padding rows (whose scales are NaN here) give zeros, the others the same bits as
    without pair_rows, and rows behind the last tile are untouched; read from the tokens,
    rows are what they are in expert order."""
    k, E, N, K = 2, 5, 160, 544
    say(f"padding rows block_m {bm} tokens {T} gather {gather}")
    g = torch.Generator().manual_seed(15)
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).int().cuda()
    al = binding.moe_lora_align(ids, torch.full((T,), -1, dtype=torch.int32, device="cuda"), None, E, 0,
                                bm, pair_rows=True)
    used, M = int(al["num_rows_padded"].cpu()[0]), al["capacity"]
    sid = al["sorted_pair_ids"]
    pad = sid >= T * k
    w, ws = int8_weights(E, N, K, 16)
    tok, tok_s = int8_rows(T, K, 17)
    at = torch.where(pad, 0, sid).long() // k
    x, xs = tok[at].contiguous(), tok_s[at].clone()
    xs[pad] = float("nan")
    plain = {n: al[n] for n in ("block_m", "tile_expert")}
    row_expert = al["tile_expert"].cpu().numpy().repeat(bm)[:M]
    row_expert = np.where(pad.cpu().numpy(), -1, row_expert)
    for silu in (False, True):
        for dt in (torch.float32, torch.bfloat16):
            mark = torch.full((M, N // 2 if silu else N), -9.5, dtype=dt, device="cuda")
            if gather:
                y = product(tok, tok_s, w, ws, al, silu, dt, mark.clone(), top_k=k)
            else:
                y = product(x, xs, w, ws, al, silu, dt, mark.clone())
            check_product(y, x, xs, w, ws, row_expert, silu)
            assert bool((y[:used][pad[:used]] == 0).all())
            assert torch.equal(y[used:], mark[used:])
            z = product(x, xs, w, ws, plain, silu, dt, mark.clone())
            assert torch.equal(y[~pad], z[~pad])


MANY = [  # block_m, tiles in use and behind them, N: past 256 workgroups
    (256, 18, 2, 4096), (256, 21, 0, 4096), (256, 31, 1, 2064), (128, 20, 3, 4096), (256, 36, 1, 1040), (128, 1, 0, 16),
    (256, 2, 1, 528), (64, 30, 2, 1040), (64, 70, 1, 272), (192, 24, 2, 1040), (192, 3, 1, 96), (16, 600, 3, 96),
    (32, 40, 1, 1056)]


@pytest.mark.parametrize("K", [208, 528])      # tiles of 64 rows, and those that block_m takes
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"b{c[0]}t{c[1]}N{c[3]}")
def test_many_tiles(case, K):
    """Row tiles with any number of rows in use, with gaps; the others give zeros."""
    bm, tiles, behind, N = case
    E, M = 3, bm * (tiles + behind)
    say(f"many tiles {case} {K}")
    g = torch.Generator().manual_seed(18)
    experts = torch.cat((torch.randint(0, E, (tiles,), generator=g), torch.full((behind,), -1)))
    fill = torch.randint(0, bm + 1, (tiles + behind,), generator=g)
    for i, n in enumerate((0, 1, 64, 65, 128, bm)[:tiles]):
        fill[i] = n
    live = torch.arange(bm).view(1, -1) < fill.view(-1, 1)
    live &= torch.rand(tiles + behind, bm, generator=g) < 0.9
    live = live.reshape(-1)
    T = 1000                                   # tokens that the rows name
    pairs = int(live.sum()) + 1
    sid = torch.full((M,), pairs, dtype=torch.int32)
    sid[live] = torch.randperm(pairs - 1, generator=g).int()
    sid[~live] = torch.where(torch.rand(int((~live).sum()), generator=g) < 0.5, -1, pairs).int()
    al = dict(block_m=bm, tile_expert=experts.int().cuda(), sorted_pair_ids=sid.cuda(), capacity=M,
              pair_rows=torch.empty(pairs, dtype=torch.int32, device="cuda"))
    w, ws = int8_weights(E, N, K, 19)
    k = (pairs + T - 1) // T
    tok, tok_s = int8_rows(T, K, 20)
    at = torch.where(live, sid, 0).long().cuda() // k
    x, xs = tok[at].contiguous(), tok_s[at].contiguous()
    row_expert = np.where(live.numpy(), experts.numpy().repeat(bm), -1)
    used = bm * tiles
    for silu in (False, True) if N % 32 == 0 else (False,):
        mark = torch.full((M, N // 2 if silu else N), -9.5, dtype=torch.bfloat16, device="cuda")
        for gather in (False, True):
            src = (tok, tok_s) if gather else (x, xs)
            y = product(*src, w, ws, al, silu, torch.bfloat16, mark.clone(), top_k=k if gather else None)
            check_product(y, x, xs, w, ws, row_expert, silu)
            assert bool((y[:used][~live[:used].cuda()] == 0).all())
            assert torch.equal(y[used:], mark[used:])


@pytest.mark.parametrize("M", [3, 40, 600])
def test_largest_sums(M):
    """The longest rows of the extreme codes: the sums reach 2^31 - 2^18 and stay integers."""
    K, N = 131056, 32
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    x[1::2, ::2] = 127
    xs, ws = torch.full((M,), 0.25, device="cuda"), torch.full((N,), 2.0, device="cuda")
    out = product(x, xs, w, ws, dt=torch.float32)
    check_product(out, x, xs, w, ws, None, False)


@pytest.mark.parametrize("M,bm", [(5, 0), (48, 16), (512, 256)])
def test_scales_that_are_not_finite(M, bm):
    """A NaN or infinite scale reaches its row or its column alone."""
    N, K, E = 96, 160, 2
    w, ws = int8_weights(E, N, K, 21)
    x, xs = int8_rows(M, K, 22)
    if bm:
        al = dict(block_m=bm, tile_expert=torch.tensor([1, 0, 1][:M // bm], dtype=torch.int32, device="cuda"))
    else:
        al, w, ws = None, w[0].contiguous(), ws[0].contiguous()
    clean = product(x, xs, w, ws, al, dt=torch.float32)
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[3] = float("nan")
    (ws2 if bm == 0 else ws2[1])[7] = float("inf")
    y = product(x, xs2, w, ws2, al, dt=torch.float32)
    of1 = torch.ones(M, dtype=torch.bool, device="cuda") if bm == 0 else al["tile_expert"].repeat_interleave(bm) == 1
    assert bool(y[3].isnan().all())
    col = y[of1, 7]
    assert not bool(col.isfinite().any())
    y[of1, 7] = clean[of1, 7]
    y[3] = clean[3]
    assert torch.equal(y, clean)


def test_silu_over_its_range():
    """gate from the far negative end, where SiLU is 0, to the far positive one."""
    K, half = 16, 512
    x = torch.zeros(1, K, dtype=torch.int8, device="cuda")
    x[0, 0] = 1
    w = torch.zeros(2 * half, K, dtype=torch.int8, device="cuda")
    w[:, 0] = 1
    gate = torch.linspace(-110, 110, half)
    ws = torch.cat((gate, torch.full((half,), 3.0))).cuda()
    xs = torch.ones(1, device="cuda")
    check_product(product(x, xs, w, ws, silu=True, dt=torch.float32), x, xs, w, ws, None, True)


# ---------------------------------------------------------------------------
# a run of them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 64, 32), (64, 16, 4, 256, 96), (700, 4, 2, 128, 160)])
def test_norm_route_layer(T, E, k, H, I):
    """norm -> router -> layer, as a model has them, against the layer in 64 bits on the
    values that the integers stand for.  Beside the rounding of y it goes through one
    quantisation that the reference leaves out: an activation is off by half a step of its row,
    row maximum / 254."""
    say(f"layer {T} {E} {k} {H} {I}")
    g = torch.Generator().manual_seed(23)
    x, res = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    router = torch.randn(E, H, generator=g).cuda() * H ** -0.5
    wgu = binding.moe_lora_int8_quantize((torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).cuda())
    wd = binding.moe_lora_int8_quantize((torch.randn(E, H, I, generator=g) * I ** -0.5).cuda())
    codes, scales, h, y = binding.moe_lora_rms_norm_quantize(x, w, 1e-6, residual=res, y_dtype=torch.float32)
    ids, weights = binding.moe_lora_route((y @ router.t()).contiguous(), k)
    inputs = dict(topk_ids=ids, topk_weights=weights, w_gate_up_int8=wgu, w_down_int8=wd,
                  x_int8=(codes, scales))
    out = binding.run_int8_layer(inputs)
    assert out.dtype == torch.bfloat16 and out.shape == (T, H)
    x64 = np64(binding.moe_lora_int8_dequantize(codes, scales, out_dtype=torch.float32))
    gu64, d64 = (c.cpu().numpy().astype(np.float64) * s.cpu().numpy().astype(np.float64)[..., None]
                 for c, s in (wgu, wd))
    ref, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e, wt = int(ids[t, j]), float(weights[t, j])
            gate, up = gu64[e, :I] @ x64[t], gu64[e, I:] @ x64[t]
            act = gate / (1 + np.exp(-gate)) * up
            z = d64[e] @ act
            ref[t] += wt * z
            # act: bf16 and half a step of the quantisation (whose maximum is bf16's)
            d_act = 2.0 ** -8 * np.abs(act) * 1.01 + np.abs(act).max() * 1.01 / 254
            tol[t] += wt * (np.abs(d64[e]) @ d_act + 2.0 ** -20 * np.abs(z))
    tol += 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(np64(out) - ref) <= tol).all()
    # tokens that are quantized by the layer itself, and given block sizes
    vals = binding.moe_lora_int8_dequantize(codes, scales, out_dtype=torch.float32)
    for bm in (16, 64, 256):
        again = binding.run_int8_layer(dict(inputs, x_int8=None, x=vals), block_m=bm, out_dtype=torch.float32)
        tol1 = tol + 2 * (tol - 2.0 ** -8 * np.abs(ref))
        assert (np.abs(np64(again) - ref) <= tol1).all()


def test_run_without_gather_is_the_same():
    """Codes and scales brought into expert order by moe_lora_permute give the same bits."""
    T, E, k, H, N = 200, 6, 3, 96, 64
    g = torch.Generator().manual_seed(24)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    al = binding.moe_lora_align(ids, torch.full((T,), -1, dtype=torch.int32, device="cuda"), None, E, 0, 32,
                                pair_rows=True)
    used = int(al["num_rows_padded"].cpu()[0])
    w, ws = int8_weights(E, N, H, 25)
    codes, scales = binding.moe_lora_int8_quantize(rand((T, H), "bf16", 26))
    rows = binding.moe_lora_permute(codes.view(torch.uint8), al, k).view(torch.int8)
    rs = binding.moe_lora_permute(scales.view(T, 1), al, k).view(-1)
    a = binding.moe_lora_int8_gemm(rows, rs, w, ws, align_out=al)
    b = binding.moe_lora_int8_gemm(codes, scales, w, ws, align_out=al, top_k=k)
    assert torch.equal(a[:used], b[:used])
