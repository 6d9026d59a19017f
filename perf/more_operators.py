"""Performance cases of the operators around experts in 8-bit integers, and of the router's loss.

Four operators, each in its plain form (elementary torch operations) and as the package's own
call:

* ``norm``      h = x + residual; n = h / sqrt(mean(h^2) + eps) * weight; n in 8-bit integers under
                one scale per token, those back to values, and on request h and n themselves.
* ``quantize``  rows to 8-bit integers under one scale per row, and back to values.
* ``gemm``      x W^T per expert with x and W in 8-bit integers, a scale for each token and one for
                each output channel, optionally with SiLU(gate) * up behind it.
* ``balance``   pairs per expert and the loss E / (n k) sum_e counts_e mean_t softmax(logits_t)_e of
                the n tokens that take part, and its gradient for the logits.

The scale of a row is its largest magnitude over 127, rounded to 32 bits; an integer is the value
over that scale, to the nearest, ties to even.  Rows behind the last bucket of an expert order are
left as they are; the buffers given here hold zeros there.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, tokens, hidden, dtype, residual, y):
    return dict(op="norm", tokens=tokens, hidden=hidden, dtype=dtype, residual=residual, y=y,
                name=name)


def _quantize(name, rows, cols, dtype):
    return dict(op="quantize", rows=rows, cols=cols, dtype=dtype, name=name)


def _gemm(name, tokens, top_k, experts, n, k, gather, silu, out, block_m):
    return dict(op="gemm", tokens=tokens, top_k=top_k, experts=experts, n=n, k=k, gather=gather,
                silu=silu, out=out, block_m=block_m, name=name)


def _balance(name, tokens, experts, top_k, dtype, masked, backward):
    return dict(op="balance", tokens=tokens, experts=experts, top_k=top_k, dtype=dtype,
                masked=masked, backward=backward, name=name)


def listed():
    return [
        # in front of the widest layer, a decode step: latency
        _norm("norm decode", 128, 7168, "bf16", True, True),
        # the same of a prefill
        _norm("norm prefill", 16384, 7168, "bf16", True, True),
        # fp32 tokens of an odd width, no residual, integers alone
        _norm("norm ragged", 4097, 1001, "f32", False, False),
        # activations between the two products of a decode step (64 tokens x 8, padded)
        _quantize("quantize activations", 2432, 768, "bf16"),
        # the gate and up weights of a layer of 8 experts, once at load time
        _quantize("quantize weights", 8 * 28672, 4096, "bf16"),
        # a dense projection of one token: latency of a weight stream
        _gemm("gemm dense token", 1, 1, 0, 2112, 7168, False, False, "bf16", 16),
        # gate and up of a decode step, from the tokens: every expert's weights are read once
        _gemm("gemm decode", 64, 8, 128, 1536, 2048, True, True, "bf16", 16),
        # gate and up of a prefill on one of 8 expert-parallel ranks, rows in expert order
        _gemm("gemm prefill up", 16384, 1, 32, 4096, 7168, False, True, "bf16", 256),
        # down of a prefill of a layer of 8 wide experts, for the fp32 combine
        _gemm("gemm prefill down", 4096, 2, 8, 4096, 14336, False, False, "f32", 256),
        # loads of a decode step's experts and the loss's value: latency
        _balance("balance decode", 64, 128, 8, "f32", False, False),
        # a training step over the widest router: loss and gradient
        _balance("balance step", 16384, 256, 8, "f32", False, True),
        # padded sequences, bf16 logits, an odd number of experts, some of them switched off
        _balance("balance ragged", 4097, 61, 6, "bf16", True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "gemm", "gemm", "balance"))
    if op == "norm":
        hidden = _log(rng, 16, 16384)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        tokens = max(1, min(_log(rng, 1, 16384), 16384 * 7168 // (2 * hidden)))
        case = _norm("", tokens, hidden, rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.7,
                     rng.random() < 0.6)
    elif op == "quantize":
        cols = _log(rng, 16, 16384)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = max(1, min(_log(rng, 1, 262144), 8 * 28672 * 4096 // (2 * cols)))
        case = _quantize("", rows, cols, rng.choice(("bf16", "f32")))
    elif op == "balance":
        experts = _log(rng, 2, 512)
        top_k = rng.randint(1, min(8, max(1, experts // 2)))
        tokens = max(1, min(_log(rng, 1, 32768), 16384 * 256 // experts))
        case = _balance("", tokens, experts, top_k, rng.choice(("f32", "f32", "bf16")),
                        rng.random() < 0.5, rng.random() < 0.6)
    else:
        silu, out = rng.random() < 0.4, rng.choice(("bf16", "bf16", "f32"))
        n, k = 32 * _log(rng, 2, 200), 16 * _log(rng, 4, 640)
        if rng.random() < 0.5:
            n, k = max(128, n // 128 * 128), max(128, k // 128 * 128)
        most = 16384 * 4096 * 7168
        if rng.random() < 0.25:   # one dense weight
            tokens = max(1, min(_log(rng, 1, 8192), most // (n * k)))
            case = _gemm("", tokens, 1, 0, n, k, False, silu, out, 16)
        else:
            experts = min(_log(rng, 2, 128), max(2, 32 * 4096 * 7168 // (n * k)))
            top_k = rng.randint(1, min(8, experts))
            tokens = max(1, min(_log(rng, 1, 8192), most // (2 * n * k * top_k)))
            # the block a user takes for these sizes: about the rows of an expert, 256 at most
            per = tokens * top_k / experts
            block_m = 16 if per <= 24 else 32 if per <= 48 else 64 if per <= 128 else 128 if per <= 512 else 256
            while experts * block_m * n * k > 4 * most and block_m > 16:
                block_m //= 2
            case = _gemm("", tokens, top_k, experts, n, k, rng.random() < 0.5, silu, out, block_m)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _layout(g, tokens, top_k, experts, block_m, dev):
    """The expert-order layout of one batch, routed at random: the arrays that moe_lora_align
    writes."""
    logits = torch.randn(tokens, experts, generator=g, device=dev)
    logits += 0.3 * torch.randn(experts, generator=g, device=dev)
    key = torch.topk(logits, top_k, dim=1).indices.reshape(-1)
    pairs = tokens * top_k
    counts = torch.bincount(key, minlength=experts)
    padded = (counts + block_m - 1) // block_m * block_m
    order = torch.argsort(key, stable=True)
    first = torch.cumsum(counts, 0) - counts
    start = torch.cumsum(padded, 0) - padded
    row = start[key[order]] + torch.arange(pairs, device=dev) - first[key[order]]
    cap = pairs + min(pairs, experts) * (block_m - 1)
    cap = (cap + block_m - 1) // block_m * block_m
    sorted_ids = torch.full((cap,), pairs, dtype=torch.int32, device=dev)
    sorted_ids[row] = order.int()
    pair_rows = torch.empty(pairs, dtype=torch.int32, device=dev)
    pair_rows[order] = row.int()
    tile_expert = torch.full((cap // block_m,), -1, dtype=torch.int32, device=dev)
    used = torch.repeat_interleave(torch.arange(experts, device=dev), padded // block_m)
    tile_expert[:used.numel()] = used.int()
    return dict(sorted_pair_ids=sorted_ids, pair_rows=pair_rows, tile_expert=tile_expert,
                num_rows_padded=padded.sum().int().reshape(1), capacity=cap, block_m=block_m,
                num_pairs=pairs)


def _int8_of(x):
    """(integers, scales) of the rows of x; 64 bits decide next to a border."""
    scales = (x.abs().amax(-1).double() / 127).float()
    step = torch.where(scales > 0, scales, torch.ones_like(scales)).double().unsqueeze(-1)
    return torch.clamp(torch.round(x.double() / step), -127, 127).to(torch.int8), scales


def _tokens_like(g, rows, cols, dev):
    """Activations: rows of unlike sizes, and a few channels larger than the others."""
    x = torch.randn(rows, cols, generator=g, device=dev)
    channel = torch.rand(cols, generator=g, device=dev)
    x *= 1 + 3 * (channel < 0.02).float()
    return x * torch.exp2(torch.randn(rows, 1, generator=g, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        T, H, dt = case["tokens"], case["hidden"], DTYPES[case["dtype"]]
        s["x"] = _tokens_like(g, T, H, dev).to(dt)
        s["residual"] = (4 * _tokens_like(g, T, H, dev)).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device=dev)).to(dt)
    elif case["op"] == "quantize":
        s["x"] = torch.empty((case["rows"], case["cols"]), dtype=DTYPES[case["dtype"]], device=dev)
        some = max(1, (1 << 27) // case["cols"])
        for r in range(0, case["rows"], some):
            part = s["x"][r:r + some]
            part.copy_(_tokens_like(g, part.shape[0], case["cols"], dev))
    elif case["op"] == "gemm":
        T, E, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        codes = torch.empty((max(E, 1), n, k), dtype=torch.int8, device=dev)
        scales = torch.empty((max(E, 1), n), dtype=torch.float32, device=dev)
        for e in range(max(E, 1)):
            w = torch.randn(n, k, generator=g, device=dev) * k ** -0.5
            codes[e], scales[e] = _int8_of(w)
        s["w"], s["w_scales"] = (codes, scales) if E else (codes[0], scales[0])
        x, xs = _int8_of(_tokens_like(g, T, k, dev))
        rows = T
        s["align"] = None
        if E:
            s["align"] = _layout(g, T, case["top_k"], E, case["block_m"], dev)
            rows = s["align"]["capacity"]
            if not case["gather"]:   # rows in expert order, zeros for padding
                ids = s["align"]["sorted_pair_ids"].long()
                x = torch.cat((x, x.new_zeros(1, k)))[ids // case["top_k"]]
                xs = torch.cat((xs, xs.new_zeros(1)))[ids // case["top_k"]]
        s["x"], s["x_scales"] = x.contiguous(), xs.contiguous()
        s["out"] = torch.zeros((rows, n // 2 if case["silu"] else n), dtype=DTYPES[case["out"]],
                               device=dev)
    else:
        T, E = case["tokens"], case["experts"]
        logits = 2 * torch.randn(T, E, generator=g, device=dev)
        logits += torch.randn(E, generator=g, device=dev)
        s["mask"] = None
        if case["masked"]:
            off = torch.randperm(E, generator=g, device=dev)[:(E - case["top_k"]) // 8]
            logits[:, off] = float("-inf")                  # experts that are switched off
            length = torch.randint(0, 65, ((T + 63) // 64, 1), generator=g, device=dev)
            ahead = torch.arange(64, device=dev) < length   # sequences padded to 64 tokens
            s["mask"] = ahead.reshape(-1)[:T].contiguous()
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["ids"] = torch.topk(s["logits"].float(), case["top_k"], dim=1).indices.int()
        s["d_loss"] = 1e-2 * (1 + torch.rand(1, generator=g, device=dev))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"norm": _plain_norm, "quantize": _plain_quantize, "gemm": _plain_gemm,
            "balance": _plain_balance}[c["op"]](s, c)


def _values(codes, scales):
    return codes.float() * scales.unsqueeze(-1)


def _run_own(s, c):
    import moe_expert_layer_segment_amd as fw
    if c["op"] == "norm":
        codes, scales, residual, y = fw.moe_lora_rms_norm_quantize(
            s["x"], s["weight"], EPS, residual=s["residual"],
            y_dtype=s["x"].dtype if c["y"] else None)
        return {"values": fw.moe_lora_int8_dequantize(codes, scales, out_dtype=s["x"].dtype),
                "scales": scales, "residual": residual, "y": y}
    if c["op"] == "quantize":
        codes, scales = fw.moe_lora_int8_quantize(s["x"])
        return {"values": fw.moe_lora_int8_dequantize(codes, scales, out_dtype=s["x"].dtype),
                "scales": scales}
    if c["op"] == "gemm":
        return {"out": fw.moe_lora_int8_gemm(s["x"], s["x_scales"], s["w"], s["w_scales"],
                                             align_out=s["align"],
                                             top_k=c["top_k"] if c["gather"] else None,
                                             silu_mul=c["silu"], out=s["out"])}
    stats = fw.moe_lora_balance_loss(s["logits"], s["ids"], s["mask"])
    out = {"loss": stats["loss"], "counts": stats["counts"], "mean_probs": stats["mean_probs"]}
    if c["backward"]:
        out["d_logits"] = fw.moe_lora_balance_loss_backward(s["d_loss"], s["logits"], stats, s["mask"])
    return out


def _plain_norm(s, c):
    # 64 bits: the integers' borders
    h = s["x"].double()
    if c["residual"]:
        h = h + s["residual"].double()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].double()
    codes, scales = _int8_of(n)
    dt = s["x"].dtype
    return {"values": _values(codes, scales).to(dt), "scales": scales,
            "residual": h.to(dt) if c["residual"] else None, "y": n.to(dt) if c["y"] else None}


def _plain_quantize(s, c):
    some = max(1, (1 << 28) // c["cols"])
    parts = [_int8_of(s["x"][r:r + some].float()) for r in range(0, c["rows"], some)]
    return {"values": torch.cat([_values(*p).to(s["x"].dtype) for p in parts]),
            "scales": torch.cat([p[1] for p in parts])}


def _plain_gemm(s, c):
    # products of integers: exact in 32 bits while the sums stay below 2^24, which they do by far
    x, xs = s["x"], s["x_scales"].unsqueeze(-1)
    if c["experts"]:
        te, bm = s["align"]["tile_expert"].long(), c["block_m"]
        if c["gather"]:
            ids = s["align"]["sorted_pair_ids"].long()
            live = (ids < s["align"]["num_pairs"]).unsqueeze(-1)
            token = torch.clamp(ids // c["top_k"], max=c["tokens"] - 1)
            x, xs = x[token] * live, xs[token] * live
        w, ws = s["w"].float(), s["w_scales"]
        y = torch.empty((x.shape[0], c["n"]), dtype=torch.float32, device=x.device)
        some = max(1, (1 << 31) // (c["n"] * c["k"]))        # tiles at a time
        for t in range(0, te.numel(), some):
            e = te[t:t + some].clamp(min=0)
            rows = slice(t * bm, (t + e.numel()) * bm)
            part = torch.matmul(x[rows].float().reshape(-1, bm, c["k"]), w[e].transpose(1, 2))
            part = part * ws[e].unsqueeze(1) * (te[t:t + some] >= 0).reshape(-1, 1, 1)
            y[rows] = part.reshape(-1, c["n"]) * xs[rows]
    else:
        y = torch.matmul(x.float(), s["w"].float().t()) * s["w_scales"] * xs
    if c["silu"]:
        gate, up = y[:, :c["n"] // 2], y[:, c["n"] // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    return {"out": y.to(DTYPES[c["out"]])}


def _plain_balance(s, c):
    # 64 bits: sums over the tokens, and the difference in the gradient
    z = s["logits"].double()
    z = z - z.amax(-1, keepdim=True)
    p = torch.exp(z)
    p = p / p.sum(-1, keepdim=True)
    live = torch.ones(c["tokens"], device=z.device) if s["mask"] is None else s["mask"]
    live = live.double().unsqueeze(-1)
    n = live.sum()
    per = 1 / torch.clamp(n, min=1)
    p = p * live
    hits = s["ids"].unsqueeze(-1) == torch.arange(c["experts"], device=z.device, dtype=torch.int32)
    counts = (hits.sum(1) * live.to(torch.int64)).sum(0)
    mean = p.sum(0) * per
    factor = c["experts"] / c["top_k"] * per
    out = {"loss": (factor * (counts * mean).sum()).float().reshape(1), "counts": counts.int(),
           "mean_probs": mean.float()}
    if c["backward"]:
        inner = counts - (counts * p).sum(-1, keepdim=True)
        out["d_logits"] = (s["d_loss"].double() * factor * per * p * inner).to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "norm":
        n, es = case["tokens"] * case["hidden"], size[case["dtype"]]
        moved = 2 + 2 * case["residual"] + case["y"]
        return {"bytes": n * (es * moved + 2) + 8 * case["tokens"] + es * case["hidden"],
                "flops": 8 * n}
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * (size[case["dtype"]] + 1) + 8 * case["rows"], "flops": 4 * n}
    if case["op"] == "gemm":
        pairs = case["tokens"] * case["top_k"]
        n, k, E = case["n"], case["k"], case["experts"]
        touched = E * (1 - (1 - 1 / E) ** pairs) if E > 1 else 1   # experts with a row, routed evenly
        out = (n // 2 if case["silu"] else n) * size[case["out"]]
        x = (case["tokens"] if case["gather"] else pairs) * (k + 4)
        return {"bytes": touched * n * (k + 4) + x + pairs * out, "flops": 2 * pairs * n * k}
    T, E = case["tokens"], case["experts"]
    once = T * E * size[case["dtype"]]
    moved = once + 4 * T * case["top_k"] + 8 * E + (T if case["masked"] else 0)
    if case["backward"]:
        moved += once          # the logits were read once already
    return {"bytes": moved, "flops": T * E * (9 if case["backward"] else 4)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _held64(v):
    """The values that rows of float64 values are held as, under 32-bit scales."""
    step = (v.abs().amax(1) / 127.0).to(torch.float32)
    divisor = step.double()
    divisor[divisor == 0] = 1.0
    return (v / divisor[:, None]).round().clamp(-127, 127) * step.double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h += s["residual"].double()
        rms = (h.square().sum(1) / case["hidden"] + EPS).sqrt()
        n = s["weight"].double() * (h / rms[:, None])
        return {"values": _held64(n), "scales": n.abs().amax(1) / 127.0,
                "residual": h if case["residual"] else None, "y": n if case["y"] else None}
    if case["op"] == "quantize":
        values = torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device)
        scales = torch.empty(case["rows"], dtype=torch.float64, device=s["x"].device)
        some = max(1, (1 << 26) // case["cols"])
        for r in range(0, case["rows"], some):
            x = s["x"][r:r + some].double()
            values[r:r + some] = _held64(x)
            scales[r:r + some] = x.abs().amax(1) / 127.0
        return {"values": values, "scales": scales}
    if case["op"] == "gemm":
        n, E = case["n"], case["experts"]
        x = s["x"].double() * s["x_scales"].double()[:, None]
        if E:
            row_expert = s["align"]["tile_expert"].repeat_interleave(case["block_m"])
            ids = s["align"]["sorted_pair_ids"].long()
            y = torch.zeros((ids.numel(), n), dtype=torch.float64, device=x.device)
            for e in range(E):
                at = ((row_expert == e) & (ids < s["align"]["num_pairs"])).nonzero().flatten()
                mine = x[ids[at] // case["top_k"]] if case["gather"] else x[at]
                y[at] = mine @ (s["w"][e].double() * s["w_scales"][e].double()[:, None]).T
        else:
            y = x @ (s["w"].double() * s["w_scales"].double()[:, None]).T
        if case["silu"]:
            y = y[:, :n // 2] * torch.sigmoid(y[:, :n // 2]) * y[:, n // 2:]
        return {"out": y}
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    keep = torch.arange(T, device=s["ids"].device)
    if s["mask"] is not None:
        keep = keep[s["mask"]]
    p = torch.softmax(s["logits"][keep].double(), 1)
    counts = torch.bincount(s["ids"][keep].long().reshape(-1), minlength=E).double()
    n = max(keep.numel(), 1)
    mean = p.sum(0) / n
    out = {"loss": (E / (n * k) * torch.dot(counts, mean)).reshape(1), "counts": counts.int(),
           "mean_probs": mean}
    if case["backward"]:
        # d softmax: p_e (g_e - sum_i p_i g_i) for the gradient g_e = E counts_e / (n^2 k) of p_e
        g = s["d_loss"].double() * E * counts / (float(n) * n * k)
        d = torch.zeros((T, E), dtype=torch.float64, device=p.device)
        d[keep] = p * (g - (p @ g)[:, None])
        out["d_logits"] = d
    return out
