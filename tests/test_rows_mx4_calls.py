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
    """Without num_pairs the length of pair_rows counts; with it, pair_rows must hold them."""
    al = dlayout()
    binding.moe_lora_permute(dev(4, 8), al, 2)
    assert recorder.args("moe_lora_permute")[:2] == [4, 2]
    with pytest.raises(ValueError):
        binding.moe_lora_permute(dev(5, 8), dict(al, num_pairs=10), 2)


def test_a_reused_layout_keeps_no_pair_rows_of_another_batch(recorder):
    """align without pair_rows into a layout that has them writes them, too."""
    al = align(6, 2, pair_rows=True)
    recorder.calls.clear()
    assert align(4, 2, out=al) is al
    assert recorder.args("moe_lora_align_pair_rows")[13].value == al["pair_rows"].data_ptr()
    assert al["num_pairs"] == 8
    with pytest.raises(ValueError):
        align(4, 2, out=dict(al, pair_rows=i32(7)))
    recorder.calls.clear()
    assert "pair_rows" not in align(4, 2)
    recorder.args("moe_lora_align")
