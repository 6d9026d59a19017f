"""The rows-in-expert-order and MX4 calls without a GPU: exported symbols, the
ctypes struct against the C one, refusals of the C ABI before any device work,
refusals of the binding, and the oracle's own pins."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import rows_mx4_oracle as ro
from moe_expert_layer_segment_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1001)
F32, BF16, FP8, U8, MX4 = 0, 1, 2, 3, 4
OK, INVALID, UNSUPPORTED = binding.OK, binding.ERR_INVALID, binding.ERR_UNSUPPORTED

CALLS = ("moe_lora_align_pair_rows", "moe_lora_permute", "moe_lora_permute_backward",
         "moe_lora_unpermute", "moe_lora_unpermute_backward", "moe_lora_mx4_quantize",
         "moe_lora_mx4_dequantize", "moe_lora_mx4_gemm")


@pytest.mark.parametrize("load", [binding.lib, binding.debug_lib])
def test_calls_are_exported(load):
    assert all(hasattr(load(), n) for n in CALLS)
    with open(os.path.join(ROOT, "include", "moe_lora.h")) as f:
        src = f.read()
    assert all(f"int {n}(" in src for n in CALLS)


def test_gemm_args_layout_matches_c(tmp_path):
    fields = [f[0] for f in binding.Mx4GemmArgs._fields_]
    body = "\n".join(f'  printf("{n} %zu\\n", offsetof(moe_lora_mx4_gemm_args, {n}));' for n in fields)
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_lora.h"\nint main(void) {\n'
                    '  printf("size %zu\\n", sizeof(moe_lora_mx4_gemm_args));\n' + body +
                    '\n  printf("u8 %d\\nmx4 %d\\n", MOE_LORA_U8, MOE_LORA_MX4);\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)],
                   check=True)
    got = dict(line.split() for line in
               subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
               if line.strip())
    assert int(got["size"]) == ctypes.sizeof(binding.Mx4GemmArgs)
    assert int(got["u8"]) == binding.DTYPE_U8 and int(got["mx4"]) == binding.DTYPE_MX4
    for n in fields:
        assert int(got[n]) == getattr(binding.Mx4GemmArgs, n).offset, n


def test_align_pair_rows_codes():
    f = binding.lib().moe_lora_align_pair_rows
    a = [FAKE] * 8
    assert f(4, 2, 8, 2, 16, *a, None, FAKE, 1 << 30, None) == INVALID          # no pair_rows
    assert f(4, 2, 8, 2, 15, *a, FAKE, FAKE, 1 << 30, None) == INVALID          # as align
    assert f(4, 9, 8, 2, 16, *a, FAKE, FAKE, 1 << 30, None) == INVALID
    assert f(4, 2, 8, 5000, 16, *a, FAKE, FAKE, 1 << 30, None) == UNSUPPORTED
    assert f(4, 2, 8, 2, 16, *a, FAKE, FAKE, 1, None) == binding.ERR_WORKSPACE


def test_permute_codes():
    f = binding.lib().moe_lora_permute
    P = FAKE
    assert f(-1, 2, 64, BF16, 64, P, P, P, P, P, None) == INVALID
    assert f(4, 0, 64, BF16, 64, P, P, P, P, P, None) == INVALID
    assert f(4, 2, 0, BF16, 64, P, P, P, P, P, None) == INVALID
    assert f(4, 2, 64, BF16, -1, P, P, P, P, P, None) == INVALID
    assert f(4, 2, 64, FP8, 64, P, P, P, P, P, None) == UNSUPPORTED
    assert f(4, 2, 64, MX4, 64, P, P, P, P, P, None) == UNSUPPORTED
    assert f(1 << 29, 2, 64, BF16, 64, P, P, P, P, P, None) == UNSUPPORTED      # pairs
    assert f(4, 2, (1 << 24) + 1, BF16, 64, P, P, P, P, P, None) == UNSUPPORTED
    assert f(4, 2, 64, BF16, 1 << 31, P, P, P, P, P, None) == UNSUPPORTED
    for i in range(5):
        args = [P] * 5
        args[i] = None
        assert f(4, 2, 64, BF16, 64, *args, None) == INVALID, i
    assert f(4, 2, 64, BF16, 64, ODD, P, P, P, P, None) == INVALID              # not element-aligned
    assert f(4, 2, 64, F32, 64, P, P, P, P, ctypes.c_void_p(0x1002), None) == INVALID
    assert f(4, 2, 64, U8, 0, None, None, FAKE, None, None, None) == OK         # no rows: nothing to do


def test_unpermute_codes():
    lib = binding.lib()
    f, b, g = lib.moe_lora_unpermute, lib.moe_lora_permute_backward, lib.moe_lora_unpermute_backward
    P = FAKE
    assert f(4, 2, 64, U8, U8, 64, P, P, P, P, None) == UNSUPPORTED
    assert f(4, 2, 64, BF16, MX4, 64, P, P, P, P, None) == UNSUPPORTED
    assert f(4, -2, 64, BF16, BF16, 64, P, P, P, P, None) == INVALID
    assert f(4, 2, 64, BF16, BF16, 64, None, P, P, P, None) == INVALID
    assert f(4, 2, 64, BF16, BF16, 64, P, None, P, P, None) == INVALID
    assert f(4, 2, 64, BF16, BF16, 64, P, P, P, None, None) == INVALID
    assert f(4, 2, 64, BF16, BF16, 64, P, P, P, ODD, None) == INVALID
    assert f(0, 2, 64, BF16, BF16, 64, None, None, None, None, None) == OK
    assert b(4, 2, 64, BF16, FP8, 64, P, P, P, None) == UNSUPPORTED
    assert b(4, 2, 64, BF16, F32, 64, P, None, P, None) == INVALID
    assert b(0, 2, 64, BF16, F32, 64, None, None, None, None) == OK
    ok = [P] * 8
    assert g(4, 2, 64, U8, BF16, 64, *ok, None) == UNSUPPORTED
    assert g(4, 2, 64, BF16, 9, 64, *ok, None) == UNSUPPORTED
    for i in (0, 1, 2, 3, 4, 5, 6):   # dy, rows, layout arrays, weights, d_rows
        args = list(ok)
        args[i] = None
        assert g(4, 2, 64, BF16, BF16, 64, *args, None) == INVALID, i
    assert g(4, 2, 64, BF16, F32, 64, ctypes.c_void_p(0x1002), *ok[1:], None) == INVALID
    assert g(0, 2, 64, BF16, BF16, 0, *[None] * 8, None) == OK


def test_mx4_codes():
    lib = binding.lib()
    q, d = lib.moe_lora_mx4_quantize, lib.moe_lora_mx4_dequantize
    P = FAKE
    assert q(-1, 64, BF16, P, None, P, P, None) == INVALID
    assert q(4, 0, BF16, P, None, P, P, None) == INVALID
    assert q(4, 48, BF16, P, None, P, P, None) == UNSUPPORTED
    assert q(4, 64, U8, P, None, P, P, None) == UNSUPPORTED
    assert q(1 << 40, 64, BF16, P, None, P, P, None) == UNSUPPORTED
    for i in (0, 2, 3):
        args = [P, None, P, P]
        args[i] = None
        assert q(4, 64, BF16, *args, None) == INVALID
    assert q(4, 64, BF16, ctypes.c_void_p(0x1008), None, P, P, None) == INVALID
    assert q(0, 64, BF16, None, None, None, None, None) == OK
    assert d(4, 33, F32, P, P, P, None) == UNSUPPORTED
    assert d(4, 64, FP8, P, P, P, None) == UNSUPPORTED
    for i in range(3):
        args = [P] * 3
        args[i] = None
        assert d(4, 64, F32, *args, None) == INVALID
    assert d(4, 64, F32, P, P, ctypes.c_void_p(0x1004), None) == INVALID
    assert d(0, 64, F32, None, None, None, None) == OK


def _gargs(**over):
    a = binding.Mx4GemmArgs()
    a.struct_size = ctypes.sizeof(binding.Mx4GemmArgs)
    a.x_dtype, a.out_dtype = MX4, BF16
    a.num_rows, a.out_features, a.in_features, a.num_experts, a.block_m = 64, 96, 64, 4, 16
    a.x = a.x_scale = a.w = a.w_scale = a.tile_expert = a.out = 0x1000
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_gemm_codes():
    call = lambda **o: binding.lib().moe_lora_mx4_gemm(ctypes.byref(_gargs(**o)), None)  # noqa: E731
    assert binding.lib().moe_lora_mx4_gemm(None, None) == INVALID
    assert call(struct_size=8) == INVALID
    assert call(x_dtype=F32) == UNSUPPORTED
    assert call(out_dtype=MX4) == UNSUPPORTED
    assert call(num_rows=-16) == INVALID
    assert call(out_features=0) == INVALID
    assert call(in_features=0) == INVALID
    assert call(num_experts=0) == INVALID
    assert call(in_features=48) == UNSUPPORTED
    assert call(out_features=40) == UNSUPPORTED
    assert call(out_features=48, silu_mul=1) == UNSUPPORTED
    assert call(in_features=(1 << 24) + 32) == UNSUPPORTED
    assert call(num_rows=1 << 30, out_features=1 << 14) == UNSUPPORTED
    assert call(block_m=24) == INVALID
    assert call(num_rows=72) == INVALID                      # not whole tiles
    assert call(tile_expert=None) == INVALID                 # four experts, no tiles
    assert call(tile_expert=None, num_experts=1, sorted_pair_ids=0x1000) == INVALID
    assert call(sorted_pair_ids=0x1000, num_pairs=-1) == INVALID
    assert call(in_features=1 << 20, out_features=1 << 17) == UNSUPPORTED   # scales of 4 GiB
    for n in ("x", "x_scale", "w", "w_scale", "out"):
        assert call(**{n: None}) == INVALID, n
    for n in ("x", "w", "out"):
        assert call(**{n: 0x1008}) == INVALID, n
    assert call(num_rows=0) == OK
    assert call(num_rows=0, tile_expert=None, num_experts=1) == OK


def _layout(T=4, k=2, cap=64):
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    return dict(sorted_pair_ids=i(cap), tile_expert=i(cap // 16), num_rows_padded=i(1),
                pair_rows=i(T * k), capacity=cap, block_m=16)


def test_binding_refuses_host_tensors_and_bad_types():
    al = _layout()
    for f in (lambda: binding.moe_lora_permute(torch.zeros(4, 8), al, 2),
              lambda: binding.moe_lora_permute_backward(torch.zeros(64, 8), al, 2),
              lambda: binding.moe_lora_unpermute(torch.zeros(64, 8), al, 2),
              lambda: binding.moe_lora_unpermute_backward(torch.zeros(4, 8), None, al, 2),
              lambda: binding.moe_lora_mx4_quantize(torch.zeros(4, 64)),
              lambda: binding.moe_lora_mx4_dequantize(torch.zeros(4, 16, dtype=torch.uint8),
                                                      torch.zeros(4, 1, dtype=torch.uint8)),
              lambda: binding.moe_lora_mx4_gemm(torch.zeros(4, 32).bfloat16(),
                                                torch.zeros(16, 16, dtype=torch.uint8),
                                                torch.zeros(16, 1, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        binding.moe_lora_permute([1, 2], al, 2)
    with pytest.raises(ValueError):
        binding.run_mx4_layer({}, activations="fp8")


class _Dev(torch.Tensor):
    """A host tensor that says it lives on a device: the binding's checks run on it
    and end before any pointer is used."""
    @property
    def is_cuda(self):
        return True


def dev(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Dev)


def dlayout(**kw):
    return {n: v.as_subclass(_Dev) if isinstance(v, torch.Tensor) else v for n, v in _layout(**kw).items()}


def test_binding_refuses_mismatched_layouts():
    al = dlayout()
    bad = pytest.raises((ValueError, TypeError))
    u8 = torch.uint8
    with bad:
        binding.moe_lora_permute(dev(4, 8), {n: v for n, v in al.items() if n != "pair_rows"}, 2)
    with bad:
        binding.moe_lora_permute(dev(5, 8), al, 2)                      # tokens
    with bad:
        binding.moe_lora_permute(dev(4, 8), al, 3)                      # top_k
    with bad:
        binding.moe_lora_permute(dev(4, 8, 2), al, 2)
    with bad:
        binding.moe_lora_permute(dev(4, 16)[:, ::2], al, 2)             # strided
    with bad:
        binding.moe_lora_permute(dev(4, 8, dtype=torch.float16), al, 2)
    with bad:
        binding.moe_lora_permute(dev(4, 8), al, 2, out=dev(60, 8))
    with bad:
        binding.moe_lora_permute(dev(4, 8), al, 2, out=dev(64, 8, dtype=torch.bfloat16))
    buf = dev(80, 8)
    with bad:
        binding.moe_lora_permute(buf[2:6], al, 2, out=buf[:64])         # overlap
    with bad:
        binding.moe_lora_unpermute(dev(60, 8), al, 2)                   # rows
    with bad:
        binding.moe_lora_unpermute(dev(64, 8), al, 2, dev(4, 3))        # weights
    with bad:
        binding.moe_lora_unpermute(dev(64, 8), al, 2, dev(4, 2, dtype=torch.bfloat16))
    with bad:
        binding.moe_lora_unpermute(dev(64, 8), al, 2, y=dev(4, 9))
    with bad:
        binding.moe_lora_unpermute(dev(64, 8), al, 2, y=dev(4, 8), out_dtype=torch.bfloat16)
    with bad:
        binding.moe_lora_unpermute(dev(64, 8, dtype=u8), al, 2)
    with bad:
        binding.moe_lora_permute_backward(dev(64, 8), al, 2, dx=dev(3, 8))
    with bad:
        binding.moe_lora_unpermute_backward(dev(4, 8), dev(64, 9), al, 2, dev(4, 2))
    with bad:
        binding.moe_lora_unpermute_backward(dev(4, 8), None, al, 2, dev(4, 2), d_weights=dev(4, 2))
    rows = dev(64, 8)
    with bad:
        binding.moe_lora_unpermute_backward(dev(4, 8), rows, al, 2, dev(4, 2), d_rows=rows)
    with bad:
        binding.moe_lora_unpermute_backward(dev(3, 8), rows, al, 2, dev(4, 2))


def test_binding_refuses_mismatched_mx4():
    bad = pytest.raises((ValueError, TypeError))
    u8, bf = torch.uint8, torch.bfloat16
    with bad:
        binding.moe_lora_mx4_quantize(dev(4, 48))
    with bad:
        binding.moe_lora_mx4_quantize(dev(4, 64, dtype=torch.float16))
    with bad:
        binding.moe_lora_mx4_quantize(dev(4, 64), codes=dev(4, 31, dtype=u8))
    with bad:
        binding.moe_lora_mx4_quantize(dev(4, 64), codes=dev(3, 32, dtype=u8), scales=dev(3, 2, dtype=u8))
    with bad:
        binding.moe_lora_mx4_quantize(dev(4, 64), num_rows_used=dev(1))
    with bad:
        binding.moe_lora_mx4_dequantize(dev(4, 32, dtype=u8), dev(4, 1, dtype=u8))
    with bad:
        binding.moe_lora_mx4_dequantize(dev(4, 32, dtype=u8), dev(4, 2, dtype=u8), out=dev(4, 63))
    w, ws = dev(4, 64, 32, dtype=u8), dev(4, 64, 2, dtype=u8)
    al = dlayout()
    x = dev(64, 64, dtype=bf)
    with bad:
        binding.moe_lora_mx4_gemm(x, w, ws)                                     # experts without tiles
    with bad:
        binding.moe_lora_mx4_gemm(x, w[0], ws[0], align_out=al)
    with bad:
        binding.moe_lora_mx4_gemm(dev(60, 64, dtype=bf), w, ws, align_out=al)   # whole tiles
    with bad:
        binding.moe_lora_mx4_gemm(dev(128, 64, dtype=bf), w, ws, align_out=al)  # more than the layout
    with bad:
        binding.moe_lora_mx4_gemm(dev(64, 96, dtype=bf), w, ws, align_out=al)
    with bad:
        binding.moe_lora_mx4_gemm(dev(64, 64), w, ws, align_out=al)             # fp32 x
    with bad:
        binding.moe_lora_mx4_gemm(dev(64, 32, dtype=u8), w, ws, align_out=al)   # codes without scales
    with bad:
        binding.moe_lora_mx4_gemm(x, w, ws, align_out=al, out=dev(64, 65, dtype=bf))
    with bad:
        binding.moe_lora_mx4_gemm(x, w, ws, align_out=al, out=dev(64, 64, dtype=torch.float16))


def test_block_m_rule():
    assert binding.mx4_block_m(64, 8, 128) == 16
    assert binding.mx4_block_m(16384, 1, 32) == 128
    assert binding.mx4_block_m(4096, 2, 8) == 256
    for T in (1, 100, 10000):
        for E in (1, 8, 256):
            assert binding.mx4_block_m(T, 2, E) in (16, 32, 64, 128, 256)


def test_oracle_pins():
    """The oracle on values worked out by hand."""
    x = np.zeros(32)
    x[:12] = [6.0, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, -0.74, 5.01, -7.9]
    codes, scales = ro.mx4_quantize(x)
    assert scales.tolist() == [127]                       # 4 <= 7.9 < 8: exponent 2, less 2
    v = ro.mx4_values(codes, scales)
    assert v[:12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0.5, -0.5, 6, -6]
    assert (codes[0] & 15, codes[0] >> 4) == (7, 8)       # even column in the low half; -0.25 -> -0
    codes, scales = ro.mx4_quantize(x * 2.0 ** -20)
    assert scales.tolist() == [107] and np.array_equal(ro.mx4_values(codes, scales), v * 2.0 ** -20)
    assert ro.mx4_quantize(np.zeros(32))[1].tolist() == [0]
    codes, scales = ro.mx4_quantize(np.where(np.arange(64) == 40, np.inf, 1.0))
    assert scales.tolist() == [125, 255] and not codes[16:].any()
    assert np.isnan(ro.mx4_values(codes, scales)[32:]).all()
    # a batch of two tokens, two pairs each; pair 2 has no row
    pr = ro.pair_rows_of([3, 9, 0, 1], 4)
    assert pr.tolist() == [2, 3, -1, 0]
    rows, written = ro.permute(np.array([[1.0], [2.0]]), pr, 2, 5)
    assert rows.ravel().tolist() == [2, 0, 1, 1, 0] and written.tolist() == [True, False, True, True, False]
    y, _ = ro.unpermute(np.array([[5.0], [0], [7], [11], [0]]), pr, 2, [[1, 2], [3, 4]])
    assert y.ravel().tolist() == [29, 20]
    d, dw, _ = ro.unpermute_backward(np.array([[2.0], [3.0]]), np.array([[5.0], [0], [7], [11], [0]]), pr, 2,
                                     [[1, 2], [3, 4]], 5)
    assert d.ravel().tolist() == [12, 0, 2, 4, 0] and dw.tolist() == [[14, 22], [0, 15]]
    out, _ = ro.mx4_gemm(np.array([[1.0, 2.0]]), np.array([[[1.0, 1], [2, 0]]]), [0], False)
    assert out.tolist() == [[3, 2]]


def test_kernels_use_no_scratch(tmp_path):
    from test_build_resources import HAVE_HIPCC, _resources
    if not HAVE_HIPCC:
        pytest.skip("hipcc missing")
    for src in ("rows.hip", "mx4.hip", "mx4_gemm.hip"):
        for name, r in _resources(src, tmp_path).items():
            assert r["scratch"] == 0 and r["spill"] == 0, (src, name, r)
