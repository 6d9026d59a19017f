"""What the binding of the rows-in-expert-order and MX4 calls passes to the library,
without a GPU: the library is replaced by one that records its calls."""
import ctypes

import pytest
import torch

from moe_expert_layer_segment_amd import binding
from test_rows_mx4_api import _Dev, dev, dlayout


class Recorder:
    """Stands in for the library: every call succeeds and is kept with its arguments
    (of a struct passed by reference, a copy)."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name in ("moe_lora_align_capacity_rows", "moe_lora_align_workspace_bytes"):
            return getattr(REAL, name)

        def call(*args):
            args = [type(a._obj).from_buffer_copy(a._obj) if hasattr(a, "_obj") else a for a in args]
            self.calls.append((name, args))
            return binding.OK
        return call

    def args(self, name):
        found = [a for n, a in self.calls if n == name]
        assert len(found) == 1, self.calls
        return found[0]


REAL = binding.lib()


@pytest.fixture
def recorder(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(binding, "lib", lambda: rec)
    monkeypatch.setattr(binding, "_stream", lambda *a: ctypes.c_void_p(0))
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)   # the index of a host tensor
    for name in ("empty", "full"):   # what the binding allocates says it is on a device, too
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, make=make, **kw: make(*a, **kw).as_subclass(_Dev))
    return rec


def i32(*shape):
    return dev(*shape, dtype=torch.int32)


def align(T, k, E=8, block_m=16, **kw):
    return binding.moe_lora_align(i32(T, k), i32(max(T, 1)), None, E, 0, block_m, **kw)


def buffers(T, k, E=8, block_m=16):
    """Buffers for the largest batch, T tokens."""
    cap = binding.moe_lora_align_capacity_rows(T, k, E, 0, block_m)
    return dict(sorted_pair_ids=i32(cap), tile_expert=i32(cap // block_m), tile_lora=i32(cap // block_m),
                expert_tile_offsets=i32(E + 1), num_rows_padded=i32(1), pair_rows=i32(T * k))


@pytest.mark.parametrize("T,k", [(64, 4), (5, 4), (1, 1), (3, 2)])
def test_larger_buffers_keep_the_batch_s_pairs(recorder, T, k):
    """Pairs are counted by the batch, not by the length of a reused pair_rows."""
    al = align(T, k, out=buffers(64, 4), pair_rows=True)
    cap = al["capacity"]
    binding.moe_lora_permute(dev(T, 32), al, k)
    assert recorder.args("moe_lora_permute")[:2] == [T, k]
    y = binding.moe_lora_unpermute(dev(cap, 32), al, k, dev(T, k))
    assert y.shape == (T, 32) and recorder.args("moe_lora_unpermute")[:2] == [T, k]
    u8 = torch.uint8
    binding.moe_lora_mx4_gemm(dev(cap, 64, dtype=torch.bfloat16), dev(8, 32, 32, dtype=u8),
                              dev(8, 32, 2, dtype=u8), align_out=al)
    assert recorder.args("moe_lora_mx4_gemm")[0].num_pairs == T * k


def test_pairs_of_a_layout_made_by_hand(recorder):
    """Without num_pairs the length of pair_rows counts, as it does where it is less."""
    al = dlayout()
    binding.moe_lora_permute(dev(4, 8), al, 2)
    assert recorder.args("moe_lora_permute")[:2] == [4, 2]
    recorder.calls.clear()
    binding.moe_lora_unpermute(dev(64, 8), dict(al, num_pairs=8, pair_rows=al["pair_rows"][:6]), 2)
    assert recorder.args("moe_lora_unpermute")[:2] == [3, 2]     # the first tokens alone
    with pytest.raises(ValueError):
        binding.moe_lora_permute(dev(5, 8), dict(al, num_pairs=10), 2)


def test_a_reused_layout_keeps_no_pair_rows_of_another_batch(recorder):
    """align without pair_rows into a layout that has them writes them, too."""
    al = align(6, 2, pair_rows=True)
    recorder.calls.clear()
    assert align(4, 2, out=al) is al
    assert recorder.args("moe_lora_align_pair_rows")[13].value == al["pair_rows"].data_ptr()
    assert al["num_pairs"] == 8
    recorder.calls.clear()
    assert "pair_rows" not in align(4, 2)
    recorder.args("moe_lora_align")
    recorder.calls.clear()
    assert "pair_rows" not in align(4, 2, out=dict(al, pair_rows=i32(7)))   # unasked, too small
    recorder.args("moe_lora_align")
    with pytest.raises(ValueError):
        align(4, 2, out=dict(al, pair_rows=i32(7)), pair_rows=True)


def mx4(E, N, K):
    return dev(E, N, K // 2, dtype=torch.uint8), dev(E, N, K // 32, dtype=torch.uint8)


def layer(T=5, k=2, E=8, H=96, I=64, **over):  # noqa: E741
    d = dict(x=dev(T, H, dtype=torch.bfloat16), topk_ids=i32(T, k), topk_weights=dev(T, k),
             w_gate_up_mx4=mx4(E, 2 * I, H), w_down_mx4=mx4(E, H, I))
    d.update(over)
    return d


@pytest.mark.parametrize("activations", ["bf16", "mx4"])
def test_mx4_layer_takes_weights_of_one_layer(recorder, activations):
    assert binding.run_mx4_layer(layer(), activations).shape == (5, 96)
    assert binding.run_mx4_layer(layer(T=0), activations).shape == (0, 96)
    assert binding.run_mx4_layer(layer(w_down_mx4=mx4(8, 128, 64)), activations).shape == (5, 128)
    assert binding.run_mx4_layer(layer(topk_weights=None), activations).shape == (5, 96)
    bad = [dict(w_down_mx4=mx4(7, 96, 64)),        # fewer experts: rows of the others stay unwritten
           dict(w_down_mx4=mx4(9, 96, 64)),
           dict(w_down_mx4=mx4(8, 96, 32)),        # another inner width
           dict(w_gate_up_mx4=mx4(8, 64, 96)),     # the gate alone
           dict(w_gate_up_mx4=mx4(8, 128, 64)),
           dict(x=dev(4, 96, dtype=torch.bfloat16)),
           dict(x=dev(5, 64, dtype=torch.bfloat16)),
           dict(w_down_mx4=tuple(t[0] for t in mx4(8, 96, 64)))]
    for over in bad:
        recorder.calls.clear()
        with pytest.raises(ValueError):
            binding.run_mx4_layer(layer(**over), activations)
        assert not recorder.calls, over


def test_calls_go_to_the_device_of_their_tensors(recorder, monkeypatch):
    """With another device current, each call switches to its tensors' and takes the
    stream that is current there."""
    entered, streams = [], []

    class Switch:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *exc):
            entered.append("left")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "device", Switch)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: streams.append(index) or 77)
    al = align(4, 2, pair_rows=True)
    align(4, 2)
    rows = binding.moe_lora_permute(dev(4, 64), al, 2)
    y = binding.moe_lora_unpermute(rows, al, 2, dev(4, 2))
    binding.moe_lora_permute_backward(rows, al, 2)
    binding.moe_lora_unpermute_backward(y, rows, al, 2, dev(4, 2))
    codes, scales = binding.moe_lora_mx4_quantize(rows)
    binding.moe_lora_mx4_dequantize(codes, scales)
    binding.moe_lora_mx4_gemm(codes, *mx4(8, 32, 64), x_scales=scales, align_out=al)
    assert len(recorder.calls) == 9
    assert entered == [None, "left"] * 9 and streams == [None] * 9     # the index of a host tensor
    assert [args[-1] for _, args in recorder.calls] == [77] * 9


def test_products_of_more_workgroups_than_a_launch_holds():
    """The streaming kernel takes 16 rows x 64 columns a workgroup of 256 threads, the groups
    of rows in sixteens from 32 of them on; threads of a launch are counted in 32 bits.  No
    call here launches: sizes are checked before the pointers, and x is missing."""
    import test_rows_mx4_api as api

    def call(rows, cols, block_m):
        a = api._gargs(num_rows=rows, out_features=cols, in_features=32, block_m=block_m, x=None)
        return binding.lib().moe_lora_mx4_gemm(ctypes.byref(a), None)

    for rows, cols, bm in ((976, 1 << 24, 16), (131088, 130896, 16), (144 * 7, 1 << 24, 144),
                           (48 * 17, 1 << 24, 48)):
        assert -(-rows // 16) * -(-cols // 64) < 1 << 24            # as they are counted
        assert -(-rows // 256) * 16 * -(-cols // 64) >= 1 << 24     # as they are launched
        assert call(rows, cols, bm) == binding.ERR_UNSUPPORTED, (rows, cols, bm)
    for rows, cols, bm in ((768, 1 << 24, 16), (131072, 130896, 16), (992, 1 << 24, 32),
                           (1056, 254200 * 64, 32), (960, 1 << 24, 64), (496, 1 << 24, 16)):
        assert call(rows, cols, bm) == binding.ERR_INVALID, (rows, cols, bm)


def over(t, *shape, dtype=torch.float32):
    """A tensor of `shape` whose memory ends inside that of `t`."""
    n = max(t.numel() * t.element_size(), 64)
    size = torch.zeros(*shape, dtype=dtype).nbytes
    both = torch.zeros(size + n, dtype=torch.uint8)
    at = size - 16      # `t` starts 16 bytes before the end of the other
    moved = both[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    return moved.as_subclass(_Dev), both[:size].view(dtype).view(*shape).as_subclass(_Dev)


@pytest.mark.parametrize("shared", ["topk_weights", "sorted_pair_ids", "pair_rows", "num_rows_padded",
                                    "tile_expert"])
def test_outputs_overlap_no_input(recorder, shared):
    """Every output against every array that the call reads beside the matrices."""
    T, k, H, bf = 4, 2, 64, torch.bfloat16
    al = align(T, k, pair_rows=True)
    cap = al["capacity"]
    w = dev(T, k)

    def check(call, *shape, dtype=torch.float32):
        moved, out = over(w if shared == "topk_weights" else al[shared], *shape, dtype=dtype)
        lay, weights = (al, moved) if shared == "topk_weights" else (dict(al, **{shared: moved}), w)
        with pytest.raises(ValueError, match="overlaps"):
            call(out, lay, weights)

    rows, tokens = dev(cap, H), dev(T, H)
    calls = {
        "permute": lambda: check(lambda o, a, _: binding.moe_lora_permute(tokens, a, k, out=o), cap, H),
        "permute_backward": lambda: check(
            lambda o, a, _: binding.moe_lora_permute_backward(rows, a, k, dx=o), T, H),
        "unpermute": lambda: check(lambda o, a, v: binding.moe_lora_unpermute(rows, a, k, v, y=o), T, H),
        "d_rows": lambda: check(lambda o, a, v: binding.moe_lora_unpermute_backward(
            tokens, rows, a, k, v, d_rows=o), cap, H),
        "d_weights": lambda: check(lambda o, a, v: binding.moe_lora_unpermute_backward(
            tokens, rows, a, k, v, d_weights=o), T, k),
        "gemm": lambda: check(lambda o, a, _: binding.moe_lora_mx4_gemm(
            dev(cap, H, dtype=bf), *mx4(8, 32, H), align_out=a, out=o), cap, 32, dtype=bf),
        "codes": lambda: check(lambda o, a, _: binding.moe_lora_mx4_quantize(
            rows, a["num_rows_padded"], codes=o), cap, H // 2, dtype=torch.uint8),
        "scales": lambda: check(lambda o, a, _: binding.moe_lora_mx4_quantize(
            rows, a["num_rows_padded"], scales=o), cap, H // 32, dtype=torch.uint8),
    }
    rowwise = {"permute", "permute_backward", "unpermute", "d_rows", "d_weights"}
    reads = {"topk_weights": {"unpermute", "d_rows", "d_weights"}, "pair_rows": rowwise,
             "sorted_pair_ids": rowwise | {"gemm"},
             "num_rows_padded": rowwise | {"codes", "scales"}, "tile_expert": {"gemm"}}[shared]
    recorder.calls.clear()
    for name in reads:
        calls[name]()
    assert not recorder.calls


def test_no_gradient_is_lost(recorder):
    """Inputs that require a gradient are refused where autograd would record the call;
    under no_grad, and in the forward of a Function, they are taken."""
    al = align(4, 2, pair_rows=True)
    cap, bf = al["capacity"], torch.bfloat16
    want = lambda *s, dtype=torch.float32: dev(*s, dtype=dtype).requires_grad_()  # noqa: E731
    tokens, rows, w = dev(4, 64), dev(cap, 64), dev(4, 2)
    calls = [
        lambda: binding.moe_lora_permute(want(4, 64), al, 2),
        lambda: binding.moe_lora_permute_backward(want(cap, 64), al, 2),
        lambda: binding.moe_lora_unpermute(want(cap, 64), al, 2, w),
        lambda: binding.moe_lora_unpermute(rows, al, 2, want(4, 2)),
        lambda: binding.moe_lora_unpermute_backward(want(4, 64), rows, al, 2, w),
        lambda: binding.moe_lora_unpermute_backward(tokens, want(cap, 64), al, 2, w),
        lambda: binding.moe_lora_unpermute_backward(tokens, rows, al, 2, want(4, 2)),
        lambda: binding.moe_lora_mx4_gemm(want(cap, 64, dtype=bf), *mx4(8, 32, 64), align_out=al),
        lambda: binding.run_mx4_layer(layer(x=want(5, 96, dtype=bf))),
        lambda: binding.run_mx4_layer(layer(x=want(5, 96, dtype=bf)), "mx4"),
        lambda: binding.run_mx4_layer(layer(topk_weights=want(5, 2)))]
    recorder.calls.clear()
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert not recorder.calls
    with torch.no_grad():
        for call in calls:
            call()
    binding.moe_lora_mx4_quantize(want(4, 64))     # of a weight, for serving: codes have no gradient

    class Permute(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return binding.moe_lora_permute(x, al, 2)

        @staticmethod
        def backward(ctx, d_rows):
            return binding.moe_lora_permute_backward(d_rows.contiguous().as_subclass(_Dev), al, 2)

    x = want(4, 64)
    recorder.calls.clear()
    Permute.apply(x).sum().backward()
    assert [n for n, _ in recorder.calls] == ["moe_lora_permute", "moe_lora_permute_backward"]
    assert x.grad.shape == x.shape


def test_every_variant_of_the_products_is_tested():
    """The GPU cases reach each kernel that the sizes choose between, with the groups of rows
    in order and in sixteens, scales in LDS and not, the last round split and not."""
    import test_gpu_mx4 as plain
    import test_gpu_rows_mx4_edges as edges
    cases = [(c[0], *c[1:], None) for c in plain.DENSE]
    cases += [(len(t) * bm, N, K, bm) for t, bm, N, K in plain.GROUPED]
    cases += [(bm * n if bm else n, N, K, bm) for bm, n, N, K in edges.VARIANTS]
    for kind in ("bf16", "mx4"):
        got = {edges.variant(M, N, K, bm, kind) for M, N, K, bm in cases}
        streams = {(v[1:4], "spread", v[4]) for v in got if v[0] == "stream"}
        streams |= {(v[1:4], "staged", v[5]) for v in got if v[0] == "stream"}
        sizes = [(1, 4, 4), (1, 2, 16), (2, 4, 4), (2, 2, 8), (4, 2, 4), (4, 2, 8)]
        assert streams == {(s, what, is_so) for s in sizes for what in ("spread", "staged")
                           for is_so in (False, True)}
        tiles = {v[1:3] for v in got if v[0] == "tile"}
        assert tiles == {(rows, split) for rows in (64, 128, 256) for split in (False, True)}
        by_dma = {(v[1], v[3]) for v in got if v[0] == "tile"}
        assert by_dma == {(rows, dma) for rows in (64, 128, 256)
                          for dma in ((False, True) if kind == "bf16" else (False,))}


def test_what_is_no_tensor_is_a_type_error(recorder):
    al = align(4, 2, pair_rows=True)
    rows, tokens, bf = dev(al["capacity"], 64), dev(4, 64), torch.bfloat16
    recorder.calls.clear()
    for call in (lambda: binding.moe_lora_permute([1], al, 2),
                 lambda: binding.moe_lora_permute_backward([1], al, 2),
                 lambda: binding.moe_lora_unpermute(rows, al, 2, [1]),
                 lambda: binding.moe_lora_unpermute_backward(tokens, [1], al, 2, dev(4, 2)),
                 lambda: binding.moe_lora_unpermute_backward(tokens, rows, al, 2, 1.0),
                 lambda: binding.moe_lora_mx4_quantize(rows, 3, codes=dev(len(rows), 32, dtype=torch.uint8)),
                 lambda: binding.moe_lora_mx4_gemm([1], *mx4(8, 32, 64), align_out=al),
                 lambda: binding.moe_lora_mx4_gemm(rows.to(bf), *mx4(8, 32, 64), align_out=al, out=1)):
        with pytest.raises(TypeError):
            call()
    assert not recorder.calls
