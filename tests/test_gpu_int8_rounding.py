"""Roundings of the 8-bit integer calls that fall on the middle of two numbers, and scales past
fp32's range."""
import torch

import pytest

from moe_expert_layer_segment_amd import binding

pytestmark = pytest.mark.gpu


def test_values_are_rounded_to_fp32_first():
    """71 times this scale is below the middle of 40.75 and 41 by less than fp32 holds: in fp32 it is
    the middle, whose even neighbour is 41."""
    codes = torch.tensor([[71, -71] * 8], dtype=torch.int8, device="cuda")
    scales = torch.tensor([float.fromhex("0x1.26c2b4p-1")], device="cuda")
    assert 71 * float(scales.cpu()[0]) < 40.875 and float(torch.tensor(71.0) * scales.cpu()[0]) == 40.875
    out = binding.moe_lora_int8_dequantize(codes, scales)
    assert out.tolist() == [[41.0, -41.0] * 8]


@pytest.mark.parametrize("H", [3, 40, 8192])
def test_norms_in_the_middle_of_two_codes(H):
    """n is 127, then k + 1/2 on the middle of two codes, under the scale 1: 1 / sqrt(9) is not a number
    of fp64, so either of the two may come out, and no other."""
    x = torch.full((2, H), 3.0, device="cuda")
    w = torch.arange(H, device="cuda") % 127 - 0.5
    w[0] = 127.0
    codes, scales, _, y = binding.moe_lora_rms_norm_quantize(x, w, 0.0, y_dtype=torch.float32)
    assert ((scales - 1).abs() <= 2.0 ** -23).all()
    assert bool(((y - w).abs() <= 2.0 ** -23 * w.abs()).all())
    assert bool((codes[:, 0] == 127).all()) and bool(((codes - w).abs()[:, 1:] == 0.5).all())


def test_norms_past_fp32():
    """One element of 16384 leaves 128 times the weight, whose 127th part is past fp32."""
    H, top = 16384, torch.finfo(torch.float32).max
    x = torch.zeros(3, H, device="cuda")
    x[:, 77] = 1.0
    x[1, 77] = -1.0
    x[2] = 1.0
    w = torch.ones(H, device="cuda")
    w[77] = top
    codes, scales, _, y = binding.moe_lora_rms_norm_quantize(x, w, 0.0, y_dtype=torch.float32)
    assert scales[:2].tolist() == [float("inf")] * 2 and not bool(codes[:2].any())
    assert y[:2, 77].tolist() == [float("inf"), -float("inf")] and int(y[:2].count_nonzero()) == 2
    assert abs(float(scales[2]) * 127 / top - 1) <= 2.0 ** -23
    assert int(codes[2, 77]) == 127 and int(codes[2].count_nonzero()) == 1
