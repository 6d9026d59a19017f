"""8-bit integers, the norm and the balance loss where a call's arguments, sizes or launches
leave the ordinary: pointers that are aligned to elements alone, sizes past one launch and past
32 bits, reused layouts, calls captured in graphs and on two streams at once, empty batches."""
import pytest
import torch

from gpu_helpers import say
from moe_expert_layer_segment_amd import binding
from test_gpu_balance import Balance, check, routed
from test_gpu_int8 import DT, check_product, check_quantize, int8_rows, int8_weights, rand
from test_gpu_rows_mx4_edges import empty_layout, no_slots, some_ids

pytestmark = pytest.mark.gpu


def odd(t, by):
    """t behind `by` elements of another buffer."""
    return torch.cat((t.new_zeros(by), t.reshape(-1)))[by:].view(t.shape)


# ---------------------------------------------------------------------------
# alignment
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [3, 9, 264, 1001, 8192, 17000])
def test_unaligned_rows_change_no_bit(H, dtype):
    say(f"unaligned rows {H} {dtype}")
    x, res, w = rand((21, H), dtype, 1), rand((21, H), dtype, 2), rand((H,), dtype, 3)
    want = binding.moe_lora_int8_quantize(x)
    norm = H <= 16384
    if norm:
        want_n = binding.moe_lora_rms_norm_quantize(x, w, 1e-5, residual=res, y_dtype=DT[dtype])
    want_v = binding.moe_lora_int8_dequantize(*want, out_dtype=DT[dtype])
    for by in (1, 3):
        codes, scales = odd(want[0], by), odd(want[1], by)
        codes.zero_(), scales.zero_()
        got = binding.moe_lora_int8_quantize(odd(x, by), codes=codes, scales=scales)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(binding.moe_lora_int8_dequantize(*got, out=odd(x, by)), want_v)
        if norm:
            got = binding.moe_lora_rms_norm_quantize(odd(x, by), odd(w, by), 1e-5, residual=odd(res, by),
                                                     residual_out=odd(x, by), y=odd(x, by), codes=codes, scales=scales)
            assert all(torch.equal(a, b) for a, b in zip(got, want_n))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E", [(5, 7), (5, 128), (700, 61), (700, 256)])
def test_unaligned_logits_change_no_bit(T, E, dtype):
    logits, ids = routed(T, E, 2, dtype, 4)
    mask = torch.arange(T, device="cuda") % 5 != 2
    want, d = check(logits, ids, mask)
    for by in (1, 3):
        got = binding.moe_lora_balance_loss(odd(logits, by), odd(ids, by), odd(mask, by))
        assert all(torch.equal(got[n], want[n]) for n in ("loss", "counts", "mean_probs", "num_valid"))
        dl = binding.moe_lora_balance_loss_backward(None, odd(logits, by), got, odd(mask, by), d_logits=odd(d, by))
        assert torch.equal(dl, d)


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
def test_rows_past_one_launch():
    """More rows than there are workgroups in any launch, of few columns."""
    R = (1 << 22) + 1037
    say("rows past one launch")
    x = torch.randint(-127, 128, (R, 3), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).float()
    x[:, 0] = 127
    codes, scales = binding.moe_lora_int8_quantize(x)
    assert torch.equal(codes.float(), x) and bool((scales == 1).all())
    assert torch.equal(binding.moe_lora_int8_dequantize(codes, scales, out_dtype=torch.float32), x)
    w = torch.ones(3, device="cuda")
    x[:] = torch.tensor([1.0, -1.0, 1.0], device="cuda")     # mean of squares 1
    codes, scales, _, y = binding.moe_lora_rms_norm_quantize(x, w, 0.0, y_dtype=torch.float32)
    assert torch.equal(y, x) and torch.equal(codes.float(), x * 127)
    assert bool((scales == torch.tensor(1 / 127).cuda()).all())


def test_values_past_32_bits():
    """More than 2^32 values: the last rows are what they are alone."""
    R, K = (1 << 20) + 77, 4104
    say("values past 32 bits")
    x = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    x[:-300] = 2.0
    x[-300:] = rand((300, K), "bf16", 6)
    codes, scales = binding.moe_lora_int8_quantize(x)
    tail = binding.moe_lora_int8_quantize(x[-300:].clone())
    check_quantize(x[-300:], *tail)
    assert torch.equal(codes[-300:], tail[0]) and torch.equal(scales[-300:], tail[1])
    assert bool((codes[:-300] == 127).all())
    out = binding.moe_lora_int8_dequantize(codes, scales)
    assert torch.equal(out[-300:], binding.moe_lora_int8_dequantize(*tail))
    del out, codes
    w = rand((K,), "bf16", 7)
    y = binding.moe_lora_rms_norm_quantize(x, w, 1e-6, y_dtype=torch.bfloat16)
    alone = binding.moe_lora_rms_norm_quantize(x[-300:].clone(), w, 1e-6, y_dtype=torch.bfloat16)
    assert torch.equal(y[0][-300:], alone[0]) and torch.equal(y[1][-300:], alone[1]) and torch.equal(y[3][-300:], alone[3])


def device_codes(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("M", [3, 70, 700])
def test_weights_past_32_bits(M):
    """One weight of 5 GB: columns at its start and end (streamed, and by tiles)."""
    N, K = 40000, 131056
    say(f"weights past 32 bits, {M} rows")
    w, ws = device_codes(N, K, seed=8), torch.rand(N, device="cuda") * 1e-4
    x, xs = device_codes(M, K, seed=9), torch.rand(M, device="cuda")
    y = binding.moe_lora_int8_gemm(x, xs, w, ws, out_dtype=torch.float32)
    rows = sorted({0, M // 2, M - 1})
    for lo in (0, 32768 - 8, N - 40):
        cols = slice(lo, lo + 40)
        check_product(y[rows][:, cols], x[rows], xs[rows], w[cols], ws[cols], None, False)


@pytest.mark.parametrize("bm", [16, 32, 64, 256])
def test_experts_and_rows_past_32_bits(bm):
    """Weights of 40 experts past 4 GiB, and rows of x past it, in place and gathered."""
    E, N, K = 40, 1024, 131056
    say(f"experts past 32 bits block_m {bm}")
    w, ws = device_codes(E, N, K, seed=10), torch.rand(E, N, device="cuda") * 1e-4
    tiles = [39, 0, 38, -1, 39]
    M = bm * len(tiles)
    al = dict(block_m=bm, tile_expert=torch.tensor(tiles, dtype=torch.int32, device="cuda"))
    x, xs = device_codes(M, K, seed=11), torch.rand(M, device="cuda")
    y = binding.moe_lora_int8_gemm(x, xs, w, ws, align_out=al, out_dtype=torch.float32)
    for t, e in enumerate(tiles):
        if e >= 0:
            at = [t * bm, t * bm + bm - 1]
            check_product(y[at][:, -16:], x[at], xs[at], w[e, -16:], ws[e, -16:], None, False)
    del w
    torch.cuda.empty_cache()
    w, ws = device_codes(2, 32, K, seed=12), torch.rand(2, 32, device="cuda") * 1e-4
    T = 32768                                   # tokens: 2^32 less 32768 * 16 bytes
    x, xs = device_codes(T, K, seed=13), torch.rand(T, device="cuda")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[T // 2:] = 1
    al = binding.moe_lora_align(ids, no_slots(T), None, 2, 0, bm, pair_rows=True)
    y = binding.moe_lora_int8_gemm(x, xs, w, ws, align_out=al, top_k=1, out_dtype=torch.float32)
    y = binding.moe_lora_unpermute(y, al, 1)
    for at, e in (([0, 1, 100], 0), ([T // 2, T - 2, T - 1], 1)):
        check_product(y[at], x[at], xs[at], w[e], ws[e], None, False)
    if bm == 16:
        return
    x = torch.cat((x, x[:2 * bm]))              # rows in place: past 2^32
    xs = torch.cat((xs, xs[:2 * bm]))
    te = torch.zeros(x.shape[0] // bm, dtype=torch.int32, device="cuda")
    te[-1] = 1
    y = binding.moe_lora_int8_gemm(x, xs, w, ws, align_out=dict(block_m=bm, tile_expert=te), out_dtype=torch.float32)
    for at, e in (([0, 5], 0), ([T, T + bm - 1], 0), ([T + bm, T + 2 * bm - 1], 1)):
        check_product(y[at], x[at], xs[at], w[e], ws[e], None, False)


VARIANTS = [  # block_m (0: one weight for all rows), blocks or rows, N, K, experts
    (16, 900, 272, 544, 9), (16, 64, 4112, 272, 2), (16, 300, 1040, 96, 40), (32, 301, 528, 800, 5),
    (32, 33, 4112, 144, 1), (48, 70, 1040, 272, 30), (80, 41, 1040, 528, 7), (96, 50, 800, 544, 3),
    (112, 40, 1040, 560, 11), (160, 30, 1040, 272, 4), (240, 30, 1040, 528, 4), (64, 130, 1040, 1040, 6),
    (128, 60, 1040, 4112, 6), (128, 100, 1040, 4112, 3), (128, 60, 1040, 1040, 6), (256, 19, 4352, 528, 4),
    (256, 70, 1040, 528, 4), (256, 34, 2064, 512, 4), (256, 1, 17 * 256, 1040, 1),
    (0, 96, 8464, 4112, 1), (0, 384, 11024, 528, 1), (0, 200, 28672, 528, 1), (0, 2049, 8192, 544, 1),
    (0, 4097, 1040, 256, 1), (0, 65, 16400, 272, 1), (0, 1000, 15888, 528, 1)]


@pytest.mark.parametrize("case", VARIANTS, ids=lambda c: "b{}n{}N{}K{}E{}".format(*c))
def test_variants(case):
    """Runs of blocks of one expert of any length, blocks without one among them, all sizes of
    tiles and parts of them: against products in 64 bits, which are exact here."""
    bm, n, N, K, E = case
    M = bm * n if bm else n
    say(f"variant {case}")
    g = torch.Generator().manual_seed(60)
    w, ws = device_codes(E, N, K, seed=61), torch.rand(E, N, device="cuda") * 1e-3
    x, xs = device_codes(M, K, seed=62), torch.rand(M, device="cuda")
    al = None
    expert = torch.zeros(M, dtype=torch.long)
    if bm:
        runs = torch.randint(1, 7, (n,), generator=g)
        te = torch.repeat_interleave(torch.randint(-1, E, (n,), generator=g), runs)[:n]
        te[-1 - n // 8:] = -1
        al = dict(block_m=bm, tile_expert=te.int().cuda())
        expert = te.repeat_interleave(bm)
    expert = expert.cuda()
    ref = torch.full((M, N), -9.5, dtype=torch.float32, device="cuda")
    for e in range(E):
        at = expert == e
        ref[at] = (x[at].double() @ w[e].double().t()).float() * xs[at, None] * ws[e]
    mark = torch.full((M, N), -9.5, dtype=torch.float32, device="cuda")
    wa, wsa = (w, ws) if bm else (w[0], ws[0])
    y = binding.moe_lora_int8_gemm(x, xs, wa, wsa, align_out=al, out=mark.clone())
    assert torch.equal(y, ref)
    if not bm:
        return
    # with padding rows: some in between, and every block's end behind a row of its own
    live = torch.rand(M, generator=g) < 0.9
    live &= torch.arange(M) % bm < torch.randint(0, bm + 1, (n,), generator=g).repeat_interleave(bm)
    pairs = int(live.sum())
    sid = torch.full((M,), pairs, dtype=torch.int32)
    sid[live] = torch.randperm(pairs, generator=g).int()
    al.update(sorted_pair_ids=sid.cuda(), pair_rows=torch.empty(pairs, dtype=torch.int32, device="cuda"), capacity=M)
    ref[((expert >= 0) & ~live.cuda())] = 0.0
    assert torch.equal(binding.moe_lora_int8_gemm(x, xs, wa, wsa, align_out=al, out=mark.clone()), ref)
    # the same rows where the tokens lie
    tok, tok_s = torch.zeros(pairs, K, dtype=torch.int8, device="cuda"), torch.ones(pairs, device="cuda")
    at = sid[live].long().cuda()
    tok[at], tok_s[at] = x[live.cuda()], xs[live.cuda()]
    y = binding.moe_lora_int8_gemm(tok, tok_s, wa, wsa, align_out=al, top_k=1, out=mark.clone())
    assert torch.equal(y, ref)


def test_tokens_of_many_rounds():
    """More tokens than the loss's workgroups take at once."""
    T, E, k = 1 << 20, 5, 2
    say("loss of many tokens")
    check(*routed(T, E, k, "bf16", 14), torch.arange(T, device="cuda") % 7 != 0)


# ---------------------------------------------------------------------------
# layouts
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bm", [16, 64, 256])
def test_layout_in_buffers_of_a_larger_batch(bm):
    k, E, N, K = 2, 5, 96, 160
    out = empty_layout(300, k, E, bm)
    w, ws = int8_weights(E, N, K, 15)
    for T in (300, 41, 1):
        say(f"larger buffers block_m {bm} T {T}")
        ids = some_ids(T, k, E, T)
        own = binding.moe_lora_align(ids, no_slots(T), None, E, 0, bm, pair_rows=True)
        al = binding.moe_lora_align(ids, no_slots(T), None, E, 0, bm, out=out, pair_rows=True)
        used = int(al["num_rows_padded"].cpu()[0])
        x, xs = int8_rows(T, K, 16)
        z, z2 = (binding.moe_lora_int8_gemm(x, xs, w, ws, align_out=a, top_k=k, silu_mul=True) for a in (al, own))
        assert torch.equal(z[:used], z2[:used])
        q, q2 = (binding.moe_lora_int8_quantize(v, al["num_rows_padded"]) for v in (z, z2))
        assert all(torch.equal(a[:used], b[:used]) for a, b in zip(q, q2))


def test_an_expert_named_twice_by_a_token():
    """Pairs of one token and one expert are each counted, and each has its row."""
    T, k, E, N, K = 50, 3, 4, 64, 48
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ids[:, 2] = 3
    w, ws = int8_weights(E, N, K, 17)
    x, xs = int8_rows(T, K, 18)
    al = binding.moe_lora_align(ids, no_slots(T), None, E, 0, 16, pair_rows=True)
    z = binding.moe_lora_int8_gemm(x, xs, w, ws, align_out=al, top_k=k, out_dtype=torch.float32)
    rows = al["pair_rows"].view(T, k).long()
    for j, e in enumerate((0, 0, 3)):
        check_product(z[rows[:, j]], x, xs, w[e], ws[e], None, False)
    logits, _ = routed(T, E, 1, "f32", 19)
    check(logits, ids)


def test_empty_batches():
    """No token at all: nothing to do, and nothing refused."""
    E, H, I = 4, 64, 32
    gu, down = int8_weights(E, 2 * I, H, 20), int8_weights(E, H, I, 21)
    none = dict(topk_ids=torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                topk_weights=torch.empty(0, 2, device="cuda"), w_gate_up_int8=gu, w_down_int8=down,
                x=torch.empty(0, H, dtype=torch.bfloat16, device="cuda"))
    assert binding.run_int8_layer(none).shape == (0, H)
    c, s, h, y = binding.moe_lora_rms_norm_quantize(none["x"], torch.ones(H, device="cuda"), residual=none["x"],
                                                    y_dtype=torch.float32)
    assert c.shape == h.shape == y.shape == (0, H) and s.shape == (0,)
    out = binding.moe_lora_int8_gemm(c, s, gu[0][0], gu[1][0], silu_mul=True)
    assert out.shape == (0, I)


# ---------------------------------------------------------------------------
# graphs and streams
# ---------------------------------------------------------------------------
def test_layer_captured_and_on_two_streams():
    """norm -> layer replayed from a graph with new tokens, experts and weights, beside its own
    eager calls on another stream, has the bits of the eager call."""
    T, E, k, H, I = 96, 8, 2, 512, 96
    say("layer in a graph, and on two streams")
    gu, down = int8_weights(E, 2 * I, H, 22), int8_weights(E, H, I, 23)
    weight = rand((H,), "bf16", 24)

    def batch(seed):
        return dict(ids=some_ids(T, k, E, seed), w=torch.rand(T, k, device="cuda"),
                    x=rand((T, H), "bf16", seed), res=rand((T, H), "bf16", seed + 1))

    def run(b):
        c, s, h, _ = binding.moe_lora_rms_norm_quantize(b["x"], weight, 1e-6, residual=b["res"])
        return h, binding.run_int8_layer(dict(topk_ids=b["ids"], topk_weights=b["w"], w_gate_up_int8=gu,
                                              w_down_int8=down, x_int8=(c, s)))
    held = batch(30)
    run(held)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                       # two graphs of the same buffers
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(held)
        graphs.append((graph, got))
    for seed in (31, 33, 35):
        new = batch(seed)
        for name, v in new.items():
            held[name].copy_(v)
        want = [t.clone() for t in run(new)]
        for graph, got in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    other = batch(40)
    want_other = [t.clone() for t in run(other)]
    torch.cuda.synchronize()
    for _ in range(4):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            got_other = run(other)
        mine = run(held)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], want))
        assert all(torch.equal(a, b) for a, b in zip(got_other, want_other))
        assert all(torch.equal(a, b) for a, b in zip(mine, want))


@pytest.mark.parametrize("T", [200, 3000])
def test_loss_captured_and_on_two_streams(T):
    """Loss and gradient in two graphs of one workspace, beside an eager call on another
    stream; an eager autograd graph of the same leaf lives on meanwhile."""
    E, k = 40, 3
    say(f"loss in graphs {T}")
    held, ids = routed(T, E, k, "f32", 50)
    ws = torch.empty(max(binding.moe_lora_balance_loss_workspace_bytes(T, E), 1), dtype=torch.uint8, device="cuda")
    mask = torch.arange(T, device="cuda") % 3 != 1
    leaf = held.clone().requires_grad_()
    alive = Balance.apply(leaf, ids, mask).sum()

    def run(logits, i):
        stats = binding.moe_lora_balance_loss(logits, i, mask, workspace=ws)
        return stats, binding.moe_lora_balance_loss_backward(None, logits, stats, mask)
    run(held, ids)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(held, ids)
        graphs.append((graph, got))
    names = ("loss", "counts", "mean_probs", "num_valid")
    side = torch.cuda.Stream()
    for seed in (51, 52, 53):
        new, new_ids = routed(T, E, k, "f32", seed)
        held.copy_(new), ids.copy_(new_ids)
        stats, d = check(new, new_ids, mask)
        torch.cuda.synchronize()
        for graph, (gs, gd) in graphs:
            graph.replay()
            with torch.cuda.stream(side):
                beside = binding.moe_lora_balance_loss(new, new_ids, mask)
            torch.cuda.synchronize()
            assert all(torch.equal(gs[n], stats[n]) and torch.equal(beside[n], stats[n]) for n in names)
            assert torch.equal(gd, d)
    alive.backward()
    first, first_ids = routed(T, E, k, "f32", 50)
    # (ids hold another batch by now, but its counts were taken in the forward pass)
    assert torch.equal(leaf.grad, check(first, first_ids, mask)[1])
