"""Performance cases of the expert-row operators and of the 4-bit microscaled (MX4) products.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the
package's own call:

* ``permute``    rows of x copied to their places in expert order (the layout of moe_lora_align:
                 buckets by expert, padded to block_m rows), and its gradient.
* ``unpermute``  y_t = sum_j w_tj z[row of pair (t, j)], and its gradients for z and w.
* ``quantize``   to MX4 (blocks of 32 e2m1 codes under one power-of-two scale) and back to values.
* ``gemm``       x W^T per expert with W in MX4 and x in bf16 or MX4, optionally with
                 SiLU(gate) * up behind it.

Rows behind the last bucket are left as they are by every operator; the buffers given here hold
zeros there.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # the magnitudes of codes 0..7; bit 3 is the sign


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _permute(name, tokens, top_k, experts, hidden, dtype, backward, shards=1, block_m=16):
    return dict(op="permute", tokens=tokens, top_k=top_k, experts=experts, hidden=hidden,
                dtype=dtype, backward=backward, shards=shards, block_m=block_m, name=name)


def _unpermute(name, tokens, top_k, experts, hidden, dtype, out, backward, shards=1, block_m=16):
    return dict(op="unpermute", tokens=tokens, top_k=top_k, experts=experts, hidden=hidden,
                dtype=dtype, out=out, backward=backward, shards=shards, block_m=block_m, name=name)


def _quantize(name, rows, cols, dtype):
    return dict(op="quantize", rows=rows, cols=cols, dtype=dtype, name=name)


def _gemm(name, tokens, top_k, experts, n, k, x, silu, out, block_m):
    return dict(op="gemm", tokens=tokens, top_k=top_k, experts=experts, n=n, k=k, x=x, silu=silu,
                out=out, block_m=block_m, name=name)


def listed():
    return [
        # a decode step of 64 requests over 128 experts: latency
        _permute("permute decode", 64, 8, 128, 2048, "bf16", False),
        # a training step over the widest layer: forward and gradient
        _permute("permute step", 16384, 8, 256, 7168, "bf16", True),
        # one of 8 expert-parallel ranks (most pairs live elsewhere), fp32, odd sizes
        _permute("permute shard ragged", 4097, 6, 32, 1001, "f32", True, shards=8),
        # the combine of a decode step of the widest layer
        _unpermute("unpermute decode", 128, 8, 256, 7168, "bf16", "bf16", False),
        # a training step of the fine-grained layer, fp32 rows summed into bf16 tokens
        _unpermute("unpermute step", 8192, 8, 128, 2048, "f32", "bf16", True),
        # activations of a decode step
        _quantize("quantize activations", 64, 7168, "bf16"),
        # the gate and up weights of a layer of 8 experts, once at load time
        _quantize("quantize weights", 8 * 28672, 4096, "bf16"),
        # a dense projection of one token: latency of a weight stream
        _gemm("gemm dense token", 1, 1, 0, 2112, 7168, "bf16", False, "bf16", 16),
        # gate and up of a decode step: every expert's weights are read once
        _gemm("gemm decode bf16", 64, 8, 128, 1536, 2048, "bf16", True, "bf16", 16),
        # down of a decode step with 4-bit activations
        _gemm("gemm decode mx4", 128, 8, 32, 7168, 2048, "mx4", False, "f32", 32),
        # gate and up of a prefill on one of 8 expert-parallel ranks, 4-bit activations
        _gemm("gemm prefill mx4", 16384, 1, 32, 4096, 7168, "mx4", True, "bf16", 256),
        # down of a prefill of a layer of 8 wide experts
        _gemm("gemm prefill bf16", 4096, 2, 8, 4096, 14336, "bf16", False, "bf16", 256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("permute", "unpermute", "quantize", "gemm", "gemm"))
    if op == "quantize":
        cols = 32 * _log(rng, 1, 448)
        rows = min(_log(rng, 1, 262144), 8 * 28672 * 4096 // cols)
        return _case_without_name(_quantize("", rows, cols, rng.choice(("bf16", "f32"))))
    if op in ("permute", "unpermute"):
        shards = rng.choice((1, 1, 1, 4, 8))
        experts = _log(rng, 2, 256)
        top_k = rng.randint(1, min(8, experts * shards))
        hidden = _log(rng, 24, 8192)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        tokens = max(1, min(_log(rng, 1, 16384), 16384 * 8 * 7168 // (2 * top_k * hidden)))
        block_m = rng.choice((16, 16, 32, 64, 128))
        backward = rng.random() < 0.6
        if op == "permute":
            return _case_without_name(_permute("", tokens, top_k, experts, hidden,
                                               rng.choice(("bf16", "f32")), backward, shards, block_m))
        return _case_without_name(_unpermute("", tokens, top_k, experts, hidden,
                                             rng.choice(("bf16", "f32")), rng.choice(("bf16", "f32")),
                                             backward, shards, block_m))
    silu = rng.random() < 0.4
    n = 32 * _log(rng, 2, 200)
    k = 32 * _log(rng, 2, 320)
    if rng.random() < 0.5:
        n, k = max(128, n // 128 * 128), max(256, k // 256 * 256)
    x, out = rng.choice(("bf16", "mx4")), rng.choice(("bf16", "bf16", "f32"))
    most = 16384 * 4096 * 7168
    if rng.random() < 0.25:   # one dense weight
        tokens = max(1, min(_log(rng, 1, 8192), most // (n * k)))
        return _case_without_name(_gemm("", tokens, 1, 0, n, k, x, silu, out, 16))
    experts = min(_log(rng, 2, 128), max(2, 32 * 4096 * 7168 // (n * k)))
    top_k = rng.randint(1, min(8, experts))
    tokens = max(1, min(_log(rng, 1, 8192), most // (2 * n * k * top_k)))
    # the block a user takes for these sizes: about the rows of an expert, 256 at most
    per = tokens * top_k / experts
    block_m = 16 if per <= 24 else 32 if per <= 48 else 64 if per <= 128 else 128 if per <= 512 else 256
    while experts * block_m * n * k > 4 * most and block_m > 16:
        block_m //= 2
    return _case_without_name(_gemm("", tokens, top_k, experts, n, k, x, silu, out, block_m))


def _case_without_name(case):
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _layout(g, tokens, top_k, experts, shards, block_m, dev):
    """Router weights and the expert-order layout of one batch: the arrays that moe_lora_align
    writes.  Of `shards` ranks the first holds experts [0, experts); pairs of the others have no
    row here."""
    logits = torch.randn(tokens, experts * shards, generator=g, device=dev)
    logits += 0.3 * torch.randn(experts * shards, generator=g, device=dev)
    top, ids = torch.topk(torch.softmax(logits, 1), top_k, dim=1)
    weights = top / top.sum(1, keepdim=True)
    pairs = tokens * top_k
    key = torch.where(ids < experts, ids, torch.full_like(ids, experts)).reshape(-1)
    counts = torch.bincount(key, minlength=experts + 1)
    padded = (counts + block_m - 1) // block_m * block_m
    padded[experts] = 0
    order = torch.argsort(key, stable=True)
    first = torch.cumsum(counts, 0) - counts
    start = torch.cumsum(padded, 0) - padded
    row = start[key[order]] + torch.arange(pairs, device=dev) - first[key[order]]
    local = key[order] < experts
    cap = pairs + min(pairs, experts) * (block_m - 1)
    cap = (cap + block_m - 1) // block_m * block_m
    sorted_ids = torch.full((cap,), pairs, dtype=torch.int32, device=dev)
    sorted_ids[row[local]] = order[local].int()
    pair_rows = torch.full((pairs,), -1, dtype=torch.int32, device=dev)
    pair_rows[order[local]] = row[local].int()
    tile_expert = torch.full((cap // block_m,), -1, dtype=torch.int32, device=dev)
    used = torch.repeat_interleave(torch.arange(experts, device=dev), padded[:experts] // block_m)
    tile_expert[:used.numel()] = used.int()
    return weights, dict(sorted_pair_ids=sorted_ids, pair_rows=pair_rows, tile_expert=tile_expert,
                         num_rows_padded=padded.sum().int().reshape(1), capacity=cap,
                         block_m=block_m)


def _mx4_of(x):
    """(codes, scales) of float values [.., K]: e2m1 codes, two a byte with the even column in the
    low half, and one biased exponent for 32 columns."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    exponent = torch.clamp(torch.frexp(amax)[1] - 3, min=-127)     # floor(log2(amax)) - 2
    exponent = torch.where(amax > 0, exponent, torch.full_like(exponent, -127))
    a = torch.ldexp(b, -exponent)
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0)).to(torch.uint8)
    code = (code + 8 * torch.signbit(a)).to(torch.uint8).reshape(*x.shape[:-1], -1, 2)
    codes = code[..., 0] | (code[..., 1] << 4)
    return codes, (exponent + 127).to(torch.uint8).squeeze(-1)


def _mx4_values(codes, scales):
    """The values that codes and scales stand for, in 32 bits (a scale of 255 stands for NaN)."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    half = torch.stack((codes & 15, codes >> 4), -1).int()
    v = lut[half].reshape(*scales.shape, 32)
    factor = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    factor = torch.where(scales == 255, torch.full_like(factor, float("nan")), factor)
    return (v * factor.unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _randn(g, shape, dtype, dev, scale=1.0):
    return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "quantize":
        x = torch.randn(case["rows"], case["cols"], generator=g, device=dev)
        # rows and columns of unlike sizes, as activations and weights have them
        x *= torch.exp2(2 * torch.randn(case["rows"], 1, generator=g, device=dev))
        s["x"] = x.to(DTYPES[case["dtype"]])
        return s
    if case["op"] == "gemm":
        E, n, k = case["experts"], case["n"], case["k"]
        codes = torch.empty((max(E, 1), n, k // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((max(E, 1), n, k // 32), dtype=torch.uint8, device=dev)
        for e in range(max(E, 1)):
            codes[e], scales[e] = _mx4_of(_randn(g, (n, k), torch.float32, dev, k ** -0.5))
        s["w_codes"], s["w_scales"] = (codes, scales) if E else (codes[0], scales[0])
        if E:
            _, s["align"] = _layout(g, case["tokens"], case["top_k"], E, 1, case["block_m"], dev)
            ids = s["align"]["sorted_pair_ids"].long()
            rows = s["align"]["capacity"]
            x = _randn(g, (case["tokens"] + 1, k), torch.float32, dev)
            x[-1] = 0                               # padding rows hold zeros
            x = x[ids // case["top_k"]]
        else:
            s["align"], rows = None, case["tokens"]
            x = _randn(g, (rows, k), torch.float32, dev)
        if case["x"] == "mx4":
            s["x"], s["x_scales"] = _mx4_of(x)
        else:
            s["x"], s["x_scales"] = x.bfloat16(), None
        s["out"] = torch.zeros((rows, n // 2 if case["silu"] else n), dtype=DTYPES[case["out"]],
                               device=dev)
        return s
    T, H, dt = case["tokens"], case["hidden"], DTYPES[case["dtype"]]
    s["weights"], s["align"] = _layout(g, T, case["top_k"], case["experts"], case["shards"],
                                       case["block_m"], dev)
    rows = s["align"]["capacity"]
    s["rows"] = _randn(g, (rows, H), dt, dev)         # gradient of the rows, or the experts' outputs
    if case["op"] == "permute":
        s["x"] = _randn(g, (T, H), dt, dev)
    elif case["backward"]:
        s["dy"] = _randn(g, (T, H), DTYPES[case["out"]], dev)
    if case["op"] == "permute" or case["backward"]:
        s["out"] = torch.zeros((rows, H), dtype=dt, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"permute": _plain_permute, "unpermute": _plain_unpermute,
            "quantize": _plain_quantize, "gemm": _plain_gemm}[c["op"]](s, c)


def _run_own(s, c):
    import moe_expert_layer_segment_amd as fw
    if c["op"] == "permute":
        rows = fw.moe_lora_permute(s["x"], s["align"], c["top_k"], out=s["out"])
        if not c["backward"]:
            return {"rows": rows}
        return {"rows": rows, "dx": fw.moe_lora_permute_backward(s["rows"], s["align"], c["top_k"])}
    if c["op"] == "unpermute":
        y = fw.moe_lora_unpermute(s["rows"], s["align"], c["top_k"], s["weights"],
                                  out_dtype=DTYPES[c["out"]])
        if not c["backward"]:
            return {"y": y}
        d_rows, d_weights = fw.moe_lora_unpermute_backward(s["dy"], s["rows"], s["align"],
                                                           c["top_k"], s["weights"],
                                                           d_rows=s["out"])
        return {"y": y, "d_rows": d_rows, "d_weights": d_weights}
    if c["op"] == "quantize":
        codes, scales = fw.moe_lora_mx4_quantize(s["x"])
        return {"scales": scales,
                "values": fw.moe_lora_mx4_dequantize(codes, scales, out_dtype=DTYPES[c["dtype"]])}
    return {"out": fw.moe_lora_mx4_gemm(s["x"], s["w_codes"], s["w_scales"], x_scales=s["x_scales"],
                                        align_out=s["align"], silu_mul=c["silu"], out=s["out"])}


def _by_pair(s, values):
    """values [rows, H] as [T, k, H] in 32 bits, with zeros for pairs that have no row."""
    c, at = s["case"], s["align"]["pair_rows"].long()
    got = values[at.clamp(min=0)].float() * (at >= 0).unsqueeze(-1)
    return got.reshape(c["tokens"], c["top_k"], c["hidden"])


def _to_rows(s, tokens, weights=None):
    """tokens [T, H] in expert order [rows, H], zeros where a row has no pair."""
    c, ids = s["case"], s["align"]["sorted_pair_ids"].long()
    live = ids < c["tokens"] * c["top_k"]
    at = torch.where(live, ids, torch.zeros_like(ids))
    got = tokens[at // c["top_k"]].float()
    if weights is not None:
        got = got * weights.reshape(-1)[at].unsqueeze(-1)
    return got * live.unsqueeze(-1)


def _plain_permute(s, c):
    dt = DTYPES[c["dtype"]]
    out = {"rows": _to_rows(s, s["x"]).to(dt)}
    if c["backward"]:
        out["dx"] = _by_pair(s, s["rows"]).sum(1).to(dt)
    return out


def _plain_unpermute(s, c):
    z, w = _by_pair(s, s["rows"]), s["weights"].unsqueeze(-1)
    out = {"y": (z * w).sum(1).to(DTYPES[c["out"]])}
    if c["backward"]:
        out["d_rows"] = _to_rows(s, s["dy"], s["weights"]).to(DTYPES[c["dtype"]])
        out["d_weights"] = (z * s["dy"].float().unsqueeze(1)).sum(-1)
    return out


def _plain_quantize(s, c):
    codes, scales = _mx4_of(s["x"])
    return {"scales": scales, "values": _mx4_values(codes, scales).to(DTYPES[c["dtype"]])}


def _plain_gemm(s, c):
    w = _mx4_values(s["w_codes"], s["w_scales"])
    x = s["x"].float() if s["x_scales"] is None else _mx4_values(s["x"], s["x_scales"])
    if c["experts"]:
        te = s["align"]["tile_expert"].long()
        x = x.reshape(te.numel(), c["block_m"], c["k"])
        y = torch.matmul(x, w[te.clamp(min=0)].transpose(1, 2)) * (te >= 0).reshape(-1, 1, 1)
        y = y.reshape(-1, c["n"])
    else:
        y = torch.matmul(x, w.t())
    if c["silu"]:
        gate, up = y[:, :c["n"] // 2], y[:, c["n"] // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    return {"out": y.to(DTYPES[c["out"]])}


# ---------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * size[case["dtype"]] + 2 * (n // 2 + n // 32), "flops": 4 * n}
    pairs = case["tokens"] * case["top_k"]
    if case["op"] == "gemm":
        n, k, E = case["n"], case["k"], case["experts"]
        touched = E * (1 - (1 - 1 / E) ** pairs) if E > 1 else 1   # experts with a row, routed evenly
        x = k * 2 if case["x"] == "bf16" else k // 2 + k // 32
        out = (n // 2 if case["silu"] else n) * size[case["out"]]
        return {"bytes": touched * n * (k // 2 + k // 32) + pairs * (x + out),
                "flops": 2 * pairs * n * k}
    T, H, es = case["tokens"], case["hidden"], size[case["dtype"]]
    local = pairs / case["shards"]
    if case["op"] == "permute":
        one = (T + local) * H * es + 4 * pairs
        return {"bytes": one * (2 if case["backward"] else 1),
                "flops": local * H if case["backward"] else 0}
    out = size[case["out"]]
    moved = (local * es + T * out) * H + 8 * pairs
    if case["backward"]:
        moved += (T * out + local * es) * H + 12 * pairs   # the rows were read once already
    return {"bytes": moved, "flops": local * H * (5 if case["backward"] else 2)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _decode64(codes, scales):
    """MX4 bytes as float64: value = +-m * 2^(scale - 127) with m from the code's two exponent
    bits and one mantissa bit."""
    nib = torch.empty((*codes.shape, 2), dtype=torch.uint8, device=codes.device)
    nib[..., 0], nib[..., 1] = codes % 16, codes // 16
    nib = nib.flatten(-2)
    exp, man = (nib // 2 % 4).double(), (nib % 2).double()
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * torch.exp2(exp - 1))
    mag = torch.where(nib >= 8, -mag, mag)
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)
    return mag * s


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        grid = torch.tensor(E2M1, dtype=torch.float64, device=s["x"].device)
        values = torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device)
        some = max(1, (1 << 26) // case["cols"])          # rows at a time
        for r in range(0, case["rows"], some):
            x = s["x"][r:r + some].double()
            blocks = x.reshape(x.shape[0], -1, 32)
            # the scale's exponent: the largest e with 2^e <= the block's largest magnitude, less 2
            e = torch.floor(torch.log2(blocks.abs().amax(2).clamp(min=2.0 ** -160))) - 2
            step = torch.exp2(e.clamp(min=-127)).unsqueeze(2)
            mag = blocks.abs() / step
            hi = torch.bucketize(mag, grid).clamp(max=7)
            lo = (hi - 1).clamp(min=0)
            down, up = mag - grid[lo], grid[hi] - mag
            pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            values[r:r + some] = (grid[pick] * torch.sign(blocks) * step).reshape(x.shape)
        return {"scales": None, "values": values}
    if case["op"] == "gemm":
        x = s["x"].double() if s["x_scales"] is None else _decode64(s["x"], s["x_scales"])
        y = torch.zeros((x.shape[0], case["n"]), dtype=torch.float64, device=x.device)
        if case["experts"]:
            row_expert = s["align"]["tile_expert"].repeat_interleave(case["block_m"])
            for e in range(case["experts"]):
                at = (row_expert == e).nonzero().flatten()
                y[at] = x[at] @ _decode64(s["w_codes"][e], s["w_scales"][e]).T
        else:
            y = x @ _decode64(s["w_codes"], s["w_scales"]).T
        if case["silu"]:
            half = case["n"] // 2
            y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
        return {"out": y}
    T, k, H = case["tokens"], case["top_k"], case["hidden"]
    rows = s["align"]["capacity"]
    at = s["align"]["pair_rows"].long().reshape(T, k)
    pad = torch.cat((s["rows"], s["rows"].new_zeros(1, H)))    # row -1 reads the zeros at the end
    if case["op"] == "permute":
        placed = torch.zeros((rows + 1, H), dtype=torch.float64, device=at.device)
        for j in range(k):
            placed[at[:, j]] = s["x"].double()
        out = {"rows": placed[:rows]}
        placed[rows] = 0
        if case["backward"]:
            total = torch.zeros((T, H), dtype=torch.float64, device=at.device)
            for j in range(k):
                total += pad[at[:, j]].double()
            out["dx"] = total
        return out
    w = s["weights"].double()
    y = torch.zeros((T, H), dtype=torch.float64, device=at.device)
    for j in range(k):
        y += w[:, j:j + 1] * pad[at[:, j]].double()
    out = {"y": y}
    if case["backward"]:
        dz = torch.zeros((rows + 1, H), dtype=torch.float64, device=at.device)
        dw = torch.zeros((T, k), dtype=torch.float64, device=at.device)
        for j in range(k):
            dz[at[:, j]] = w[:, j:j + 1] * s["dy"].double()
            dw[:, j] = (s["dy"].double() * pad[at[:, j]].double()).sum(1)
        out["d_rows"], out["d_weights"] = dz[:rows], dw
    return out
