"""The 8-bit integer, norm and balance-loss calls without a GPU: exported symbols, the
ctypes struct against the C one, refusals of the C ABI before any device work, refusals of
the binding, what the binding passes on, the oracle's own pins, and what the compiler made
of the kernels."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import int8_balance_oracle as ib
from moe_expert_layer_segment_amd import binding, build
from test_rows_mx4_api import _Dev, dev, dlayout
from test_rows_mx4_calls import REAL, Recorder, align, recorder  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1001)
F32, BF16, FP8, U8, MX4 = 0, 1, 2, 3, 4
OK, INVALID, UNSUPPORTED = binding.OK, binding.ERR_INVALID, binding.ERR_UNSUPPORTED
WORKSPACE = binding.ERR_WORKSPACE
I8, BF = torch.int8, torch.bfloat16

CALLS = ("moe_lora_int8_quantize", "moe_lora_int8_dequantize", "moe_lora_rms_norm_quantize",
         "moe_lora_int8_gemm", "moe_lora_balance_loss", "moe_lora_balance_loss_backward")


@pytest.mark.parametrize("load", [binding.lib, binding.debug_lib])
def test_calls_are_exported(load):
    assert all(hasattr(load(), n) for n in CALLS + ("moe_lora_balance_loss_workspace_bytes",))
    with open(os.path.join(ROOT, "include", "moe_lora.h")) as f:
        src = f.read()
    assert all(f"int {n}(" in src for n in CALLS)


def test_gemm_args_layout_matches_c(tmp_path):
    fields = [f[0] for f in binding.Int8GemmArgs._fields_]
    body = "\n".join(f'  printf("{n} %zu\\n", offsetof(moe_lora_int8_gemm_args, {n}));' for n in fields)
    prog, exe = tmp_path / "layout.c", tmp_path / "layout"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_lora.h"\nint main(void) {\n'
                    '  printf("size %zu\\n", sizeof(moe_lora_int8_gemm_args));\n' + body + '\n  return 0;\n}\n')
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.split("\n") if line.strip())
    assert int(got["size"]) == ctypes.sizeof(binding.Int8GemmArgs)
    for n in fields:
        assert int(got[n]) == getattr(binding.Int8GemmArgs, n).offset, n


def test_quantize_codes():
    q, d = binding.lib().moe_lora_int8_quantize, binding.lib().moe_lora_int8_dequantize
    P = FAKE
    assert q(-1, 64, BF16, P, None, P, P, None) == INVALID
    assert q(4, 0, BF16, P, None, P, P, None) == INVALID
    assert q(4, (1 << 24) + 1, BF16, P, None, P, P, None) == UNSUPPORTED
    assert q((1 << 40) // 64 + 1, 64, BF16, P, None, P, P, None) == UNSUPPORTED
    for dt in (-1, FP8, U8, MX4):
        assert q(4, 64, dt, P, None, P, P, None) == UNSUPPORTED
        assert d(4, 64, dt, P, P, P, None) == UNSUPPORTED
    for i in (0, 2, 3):
        args = [P, None, P, P]
        args[i] = None
        assert q(4, 64, BF16, *args, None) == INVALID, i
    assert q(4, 64, BF16, ODD, None, P, P, None) == INVALID
    assert q(4, 64, F32, ctypes.c_void_p(0x1002), None, P, P, None) == INVALID
    assert q(4, 64, BF16, P, None, P, ODD, None) == INVALID
    assert q(4, 64, BF16, P, ODD, P, P, None) == INVALID
    assert q(0, 64, BF16, None, None, None, None, None) == OK
    assert d(-1, 64, F32, P, P, P, None) == INVALID
    assert d(4, -3, F32, P, P, P, None) == INVALID
    for i in range(3):
        args = [P] * 3
        args[i] = None
        assert d(4, 64, F32, *args, None) == INVALID, i
    assert d(4, 64, F32, P, P, ctypes.c_void_p(0x1002), None) == INVALID
    assert d(4, 64, F32, P, ODD, P, None) == INVALID
    assert d(0, 64, F32, None, None, None, None) == OK


def test_norm_codes():
    f = binding.lib().moe_lora_rms_norm_quantize
    ok = [FAKE] * 7   # x, residual, weight, codes, scales, residual_out, y
    assert f(-1, 64, BF16, BF16, BF16, 1e-6, *ok, None) == INVALID
    assert f(4, 0, BF16, BF16, BF16, 1e-6, *ok, None) == INVALID
    assert f(4, 16385, BF16, BF16, BF16, 1e-6, *ok, None) == UNSUPPORTED
    assert f(1 << 40, 64, BF16, BF16, BF16, 1e-6, *ok, None) == UNSUPPORTED
    for bad in ((FP8, F32, F32), (F32, U8, F32), (F32, F32, MX4)):
        assert f(4, 64, *bad, 1e-6, *ok, None) == UNSUPPORTED
    for eps in (-1e-6, float("nan"), float("inf"), 1e39):
        assert f(4, 64, F32, F32, F32, eps, *ok, None) == INVALID
    for i in (0, 2, 3, 4):
        args = list(ok)
        args[i] = None
        assert f(4, 64, BF16, F32, F32, 1e-6, *args, None) == INVALID, i
    for i in (0, 1, 2, 4, 5, 6):
        args = list(ok)
        args[i] = ODD
        assert f(4, 64, BF16, BF16, BF16, 1e-6, *args, None) == INVALID, i
    assert f(0, 64, F32, BF16, 9, 0.0, *[None] * 7, None) == OK     # no y: its type says nothing


def _gargs(**over):
    a = binding.Int8GemmArgs()
    a.struct_size = ctypes.sizeof(binding.Int8GemmArgs)
    a.out_dtype = BF16
    a.num_rows, a.out_features, a.in_features, a.num_experts, a.block_m = 64, 96, 64, 4, 16
    a.x = a.x_scale = a.w = a.w_scale = a.tile_expert = a.out = 0x1000
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_gemm_codes():
    call = lambda **o: binding.lib().moe_lora_int8_gemm(ctypes.byref(_gargs(**o)), None)  # noqa: E731
    assert binding.lib().moe_lora_int8_gemm(None, None) == INVALID
    assert call(struct_size=8) == INVALID
    for dt in (-1, FP8, U8, MX4):
        assert call(out_dtype=dt) == UNSUPPORTED
    for name in ("num_rows", "out_features", "in_features", "num_experts", "top_k", "num_tokens"):
        assert call(**{name: -16}) == INVALID, name
    for name in ("out_features", "in_features", "num_experts"):
        assert call(**{name: 0}) == INVALID, name
    assert call(in_features=72) == UNSUPPORTED
    assert call(out_features=40) == UNSUPPORTED
    assert call(out_features=48, silu_mul=1) == UNSUPPORTED
    assert call(in_features=1 << 17) == UNSUPPORTED               # sums past int32
    assert call(num_rows=0, in_features=(1 << 17) - 16) == OK
    assert call(out_features=(1 << 24) + 16) == UNSUPPORTED
    assert call(num_rows=1 << 30, out_features=1 << 14) == UNSUPPORTED
    most = 16 * ((1 << 24) - 256)                            # of 64 columns
    assert call(num_rows=most + 16, out_features=64) == UNSUPPORTED
    assert call(num_rows=most, out_features=64, out=None) == INVALID
    for bm in (0, -16, 8, 24):
        assert call(block_m=bm) == INVALID, bm
    assert call(num_rows=72) == INVALID                      # not whole tiles
    assert call(tile_expert=None) == INVALID                 # four experts, no tiles
    assert call(tile_expert=None, num_experts=1, sorted_pair_ids=0x1000) == INVALID
    assert call(sorted_pair_ids=0x1000, num_pairs=-1) == INVALID
    gather = dict(sorted_pair_ids=0x1000, num_pairs=12, top_k=2, num_tokens=6, out=None)
    assert call(**gather) == INVALID                         # (out is missing)
    assert call(**dict(gather, sorted_pair_ids=None)) == INVALID
    assert call(**dict(gather, num_tokens=5)) == INVALID
    assert call(**dict(gather, num_pairs=13)) == INVALID
    assert call(**dict(gather, num_pairs=0, num_tokens=0)) == INVALID    # no token to name
    assert call(**dict(gather, num_tokens=1 << 26, in_features=64)) == UNSUPPORTED   # 4 GiB of x
    for n in ("x", "x_scale", "w", "w_scale", "out"):
        assert call(**{n: None}) == INVALID, n
    for n in ("x", "w", "out"):
        assert call(**{n: 0x1008}) == INVALID, n
    for n in ("x_scale", "w_scale", "tile_expert"):
        assert call(**{n: 0x1002}) == INVALID, n
    assert call(num_rows=0) == OK
    assert call(num_rows=0, tile_expert=None, num_experts=1) == OK


def test_balance_codes():
    lib = binding.lib()
    f, b, ws = lib.moe_lora_balance_loss, lib.moe_lora_balance_loss_backward, lib.moe_lora_balance_loss_workspace_bytes
    P = FAKE
    need = ws(1000, 64)
    assert need > 0 and ws(-1, 64) == ws(1000, 0) == ws(1000, 1025) == 0 and ws(1, 1024) == 0
    ok = [P, P, None, P, P, P, P, P]   # logits, ids, mask, loss, counts, mean_probs, num_valid, workspace
    for T, E, k, dt, want in ((-1, 64, 2, F32, INVALID), (1000, 0, 2, F32, INVALID), (1000, 64, 0, F32, INVALID),
                              (1000, 1025, 2, F32, UNSUPPORTED), (1000, 64, 2, FP8, UNSUPPORTED),
                              (1 << 28, 64, 4, F32, UNSUPPORTED)):
        assert f(T, E, k, dt, *ok, 1 << 40, None) == want
        assert b(T, E, k, dt, F32, P, None, P, P, None, P, None) == want
    for i in (0, 1, 3, 4, 5, 6):
        for bad in (None, ODD):
            args = list(ok)
            args[i] = bad
            assert f(1000, 64, 2, F32, *args, 1 << 40, None) == INVALID, (i, bad)
    assert f(1000, 64, 2, F32, *ok[:7], None, 1 << 40, None) == WORKSPACE
    assert f(1000, 64, 2, F32, *ok, need - 1, None) == WORKSPACE
    assert f(1000, 64, 2, F32, *ok[:7], ctypes.c_void_p(0x1004), 1 << 40, None) == INVALID
    assert b(1000, 64, 2, F32, MX4, P, None, P, P, None, P, None) == UNSUPPORTED
    good = [P, None, P, P, None, P]    # logits, mask, counts, num_valid, d_loss, d_logits
    for i in (0, 2, 3, 5):
        for bad in (None, ODD):
            args = list(good)
            args[i] = bad
            assert b(1000, 64, 2, BF16, BF16, *args, None) == INVALID, (i, bad)
    assert b(1000, 64, 2, BF16, BF16, *good[:4], ODD, P, None) == INVALID
    assert b(0, 64, 2, BF16, BF16, *[None] * 6, None) == OK


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
bad = pytest.raises((ValueError, TypeError))


@pytest.fixture(autouse=True)
def sizes(monkeypatch):
    """A library that records its calls is asked for sizes, too."""
    monkeypatch.setattr(Recorder, "moe_lora_balance_loss_workspace_bytes",
                        REAL.moe_lora_balance_loss_workspace_bytes, raising=False)


def leaf(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, requires_grad=True).as_subclass(_Dev)


def stats(E=8):
    return dict(counts=i32d(E), num_valid=i32d(1), top_k=2)


def i32d(*shape):
    return dev(*shape, dtype=torch.int32)


REFUSED = {
    "host x": lambda: binding.moe_lora_int8_quantize(torch.zeros(4, 8)),
    "half x": lambda: binding.moe_lora_int8_quantize(dev(4, 8, dtype=torch.float16)),
    "scalar x": lambda: binding.moe_lora_int8_quantize(dev()),
    "no columns": lambda: binding.moe_lora_int8_quantize(dev(4, 0)),
    "strided x": lambda: binding.moe_lora_int8_quantize(dev(4, 16)[:, ::2]),
    "list": lambda: binding.moe_lora_int8_quantize([1.0]),
    "rows used in fp32": lambda: binding.moe_lora_int8_quantize(dev(4, 8), dev(1)),
    "codes' shape": lambda: binding.moe_lora_int8_quantize(dev(4, 8), codes=dev(4, 9, dtype=I8)),
    "codes' type": lambda: binding.moe_lora_int8_quantize(dev(4, 8), codes=dev(4, 8, dtype=torch.uint8)),
    "scales' shape": lambda: binding.moe_lora_int8_quantize(dev(4, 8), scales=dev(3)),
    "scales' type": lambda: binding.moe_lora_int8_quantize(dev(4, 8), scales=dev(4, dtype=BF)),
    "x of a leaf": lambda: binding.moe_lora_int8_quantize(leaf(4, 8)),
    "value scales": lambda: binding.moe_lora_int8_dequantize(dev(4, 8, dtype=I8), dev(5)),
    "value codes": lambda: binding.moe_lora_int8_dequantize(dev(4, 8), dev(4)),
    "value out": lambda: binding.moe_lora_int8_dequantize(dev(4, 8, dtype=I8), dev(4), out=dev(4, 9)),
    "value out type": lambda: binding.moe_lora_int8_dequantize(dev(4, 8, dtype=I8), dev(4), out=dev(4, 8), out_dtype=BF),
    "value of a leaf": lambda: binding.moe_lora_int8_dequantize(dev(4, 8, dtype=I8), leaf(4)),
    "norm weight": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(9)),
    "norm weight type": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8, dtype=torch.float16)),
    "norm residual": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8), residual=dev(3, 8)),
    "norm residual type": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8), residual=dev(4, 8, dtype=BF)),
    "norm h alone": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8), residual_out=dev(4, 8)),
    "norm h shape": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8), residual=dev(4, 8), residual_out=dev(8, 8)),
    "norm y shape": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8), y=dev(4, 9)),
    "norm y type": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8), y_dtype=torch.float16),
    "norm of a leaf": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), leaf(8)),
    "norm residual leaf": lambda: binding.moe_lora_rms_norm_quantize(dev(4, 8), dev(8), residual=leaf(4, 8)),
    "loss ids": lambda: binding.moe_lora_balance_loss(dev(4, 8), i32d(3, 2)),
    "loss ids type": lambda: binding.moe_lora_balance_loss(dev(4, 8), dev(4, 2, dtype=torch.int64)),
    "loss mask": lambda: binding.moe_lora_balance_loss(dev(4, 8), i32d(4, 2), dev(5, dtype=torch.bool)),
    "loss mask type": lambda: binding.moe_lora_balance_loss(dev(4, 8), i32d(4, 2), i32d(4)),
    "loss of a leaf": lambda: binding.moe_lora_balance_loss(leaf(4, 8), i32d(4, 2)),
    "loss out": lambda: binding.moe_lora_balance_loss(dev(4, 8), i32d(4, 2), out=dict(counts=i32d(9))),
    "loss out type": lambda: binding.moe_lora_balance_loss(dev(4, 8), i32d(4, 2), out=dict(mean_probs=dev(8, dtype=BF))),
    "loss workspace": lambda: binding.moe_lora_balance_loss(dev(900, 8), i32d(900, 2), workspace=dev(8, dtype=torch.uint8)),
    "gradient of a leaf": lambda: binding.moe_lora_balance_loss_backward(leaf(1), dev(4, 8), stats()),
    "gradient's loss": lambda: binding.moe_lora_balance_loss_backward(dev(2), dev(4, 8), stats()),
    "gradient's counts": lambda: binding.moe_lora_balance_loss_backward(None, dev(4, 8), stats(9)),
    "gradient's shape": lambda: binding.moe_lora_balance_loss_backward(None, dev(4, 8), stats(), d_logits=dev(4, 9)),
    "gradient's type": lambda: binding.moe_lora_balance_loss_backward(None, dev(4, 8), stats(), out_dtype=torch.float16),
}


@pytest.mark.parametrize("name", REFUSED)
def test_binding_refuses(recorder, name):
    with bad:
        REFUSED[name]()
    assert not recorder.calls


def test_binding_refuses_overlaps(recorder):
    """Outputs that share memory with inputs or with each other, but a residual in place."""
    buf = dev(4 * 64)
    x = buf[:32].view(4, 8)
    raw = torch.zeros(4096, dtype=torch.uint8).as_subclass(_Dev)
    f = raw[:128].view(torch.float32).view(4, 8)
    with bad:
        binding.moe_lora_int8_quantize(f, codes=raw[100:132].view(I8).view(4, 8))
    with bad:
        binding.moe_lora_int8_quantize(x, scales=buf[30:34])
    with bad:
        binding.moe_lora_int8_quantize(dev(4, 8), codes=raw[:32].view(I8).view(4, 8),
                                       scales=raw[16:32].view(torch.float32))
    with bad:
        binding.moe_lora_int8_dequantize(raw[:32].view(I8).view(4, 8), dev(4), out=f)
    w, res = dev(8), buf[64:96].view(4, 8)
    with bad:
        binding.moe_lora_rms_norm_quantize(x, w, residual=res, residual_out=buf[68:100].view(4, 8))
    with bad:
        binding.moe_lora_rms_norm_quantize(x, w, residual=res, y=res)
    with bad:
        binding.moe_lora_rms_norm_quantize(x, w, residual=dev(4, 8), residual_out=res, y=buf[90:122].view(4, 8))
    with bad:
        binding.moe_lora_rms_norm_quantize(x, buf[40:48], residual=res, residual_out=buf[33:65].view(4, 8))
    assert not recorder.calls
    for place in (x, res):
        assert binding.moe_lora_rms_norm_quantize(x, w, residual=res, residual_out=place)[2] is place
    recorder.calls.clear()
    logits, ids = buf[:32].view(4, 8), i32d(4, 2)
    with bad:
        binding.moe_lora_balance_loss(logits, ids, out=dict(mean_probs=buf[30:38]))
    with bad:
        binding.moe_lora_balance_loss(dev(4, 8), ids, out=dict(loss=buf[3:4], mean_probs=buf[:8]))
    with bad:
        binding.moe_lora_balance_loss(f, ids, workspace=raw[64:1024])
    with bad:
        binding.moe_lora_balance_loss_backward(None, logits, stats(), d_logits=logits)
    assert not recorder.calls


def test_binding_refuses_mismatched_products(recorder):
    w, ws, al = dev(4, 64, 32, dtype=I8), dev(4, 64), dlayout()
    x, xs = dev(64, 32, dtype=I8), dev(64)
    g = binding.moe_lora_int8_gemm
    for call in (lambda: g(x, xs, w, ws),                                       # experts without tiles
                 lambda: g(x, xs, w[0], ws[0], align_out=al),
                 lambda: g(x, xs, w, dev(4, 63), align_out=al),
                 lambda: g(x, dev(63), w, ws, align_out=al),
                 lambda: g(dev(64, 48, dtype=I8), xs, w, ws, align_out=al),     # columns
                 lambda: g(dev(64, 32), xs, w, ws, align_out=al),               # fp32 codes
                 lambda: g(x, xs.to(BF).as_subclass(_Dev), w, ws, align_out=al),
                 lambda: g(dev(60, 32, dtype=I8), dev(60), w, ws, align_out=al),        # whole tiles
                 lambda: g(dev(128, 32, dtype=I8), dev(128), w, ws, align_out=al),      # more than the layout
                 lambda: g(x, xs, w[0], ws[0], top_k=2),                        # no layout
                 lambda: g(dev(3, 32, dtype=I8), dev(3), w, ws, align_out=al, top_k=2),  # 8 pairs of 3 tokens
                 lambda: g(x, xs, w, ws, align_out=al, top_k=0),
                 lambda: g(x, xs, w, ws, align_out=al, out=dev(64, 65, dtype=BF)),
                 lambda: g(x, xs, w, ws, align_out=al, out=dev(64, 64, dtype=BF), silu_mul=True),
                 lambda: g(x, xs, w, ws, align_out=al, out_dtype=torch.float16),
                 lambda: g(x, leaf(64), w, ws, align_out=al),
                 lambda: g(x, xs, w, leaf(4, 64), align_out=al)):
        with bad:
            call()
    raw = torch.zeros(1 << 16, dtype=torch.uint8).as_subclass(_Dev)
    with bad:
        g(raw[:2048].view(I8).view(64, 32), xs, w, ws, align_out=al,
          out=raw[2032:2032 + 8192].view(BF).view(64, 64))
    assert not recorder.calls


def test_layer_refuses(recorder):
    E, H, I = 4, 32, 16
    gu, down = (dev(E, 2 * I, H, dtype=I8), dev(E, 2 * I)), (dev(E, H, I, dtype=I8), dev(E, H))
    base = dict(topk_ids=i32d(3, 2), topk_weights=dev(3, 2), w_gate_up_int8=gu, w_down_int8=down, x=dev(3, H))
    for over in (dict(x=dev(4, H)), dict(x=leaf(3, H)), dict(topk_weights=leaf(3, 2)),
                 dict(x_int8=(dev(3, H, dtype=I8), leaf(3))),
                 dict(w_down_int8=(dev(E, H, H, dtype=I8), dev(E, H))),
                 dict(x_int8=(dev(2, H, dtype=I8), dev(2)))):
        with bad:
            binding.run_int8_layer(dict(base, **over))
        assert not any(name.endswith("unpermute") for name, _ in recorder.calls)


def test_what_a_product_is_called_with(recorder):
    """Pairs are counted by the batch; tokens read in place are as many as x has."""
    E, N, K = 8, 64, 32
    w, ws = dev(E, N, K, dtype=I8), dev(E, N)
    out = dict(align(64, 4, pair_rows=True))
    for T in (64, 5):
        recorder.calls.clear()
        al = align(T, 4, out=out, pair_rows=True)
        y = binding.moe_lora_int8_gemm(dev(T, K, dtype=I8), dev(T), w, ws, align_out=al, top_k=4, silu_mul=True)
        a = recorder.args("moe_lora_int8_gemm")[0]
        assert (a.num_pairs, a.top_k, a.num_tokens, a.num_rows) == (4 * T, 4, T, al["capacity"])
        assert (a.out_features, a.in_features, a.num_experts, a.silu_mul, a.out_dtype) == (N, K, E, 1, BF16)
        assert y.shape == (al["capacity"], N // 2) and a.sorted_pair_ids == al["sorted_pair_ids"].data_ptr()
    recorder.calls.clear()
    al = align(5, 4)
    cap = al["capacity"]
    binding.moe_lora_int8_gemm(dev(cap, K, dtype=I8), dev(cap), w, ws, align_out=al, out_dtype=torch.float32)
    a = recorder.args("moe_lora_int8_gemm")[0]
    assert a.sorted_pair_ids is None and (a.top_k, a.out_dtype, a.num_rows) == (0, F32, cap)
    recorder.calls.clear()
    binding.moe_lora_int8_gemm(dev(7, K, dtype=I8), dev(7), w[0], ws[0])
    a = recorder.args("moe_lora_int8_gemm")[0]
    assert a.tile_expert is None and (a.num_rows, a.num_experts, a.block_m) == (7, 1, 0)


def test_block_m_rule():
    assert [binding.int8_block_m(*a) for a in ((64, 8, 128), (64, 8, 32), (64, 8, 16), (16384, 1, 32))] == \
        [16, 32, 64, 256]
    for T in (0, 1, 100, 10000):
        for E in (1, 8, 256):
            assert binding.int8_block_m(T, 2, E) in (16, 32, 64, 256)


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def test_oracle_pins():
    """The oracle on values worked out by hand."""
    codes, scales = ib.int8_quantize(np.array([[127.0, 0.5, 1.5, -2.5, -126.5, 0.49]]))
    assert scales.tolist() == [1.0] and codes.tolist() == [[127, 0, 2, -2, -126, 0]]
    codes, scales = ib.int8_quantize(np.array([[np.inf, 1.0], [np.nan, 1.0], [0.0, -0.0], [-254.0, 3.0]]))
    assert np.isnan(scales[:2]).all() and scales[2:].tolist() == [0.0, 2.0]
    assert codes.tolist() == [[0, 0], [0, 0], [0, 0], [-127, 2]]
    h, n = ib.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0, np.array([[0.0, 0.0]]))
    assert np.allclose(n, np.array([[3.0, 8.0]]) / np.sqrt(12.5), rtol=1e-15) and h.tolist() == [[3, 4]]
    y = ib.int8_product(np.array([[1, -128]]), np.array([0.5]), np.array([[[2, 1], [0, -128]]]),
                        np.array([[1.0, 2.0]], dtype=np.float32), np.array([0]))
    assert y.tolist() == [[-63.0, 16384.0]]
    ln = np.log([[1.0, 3.0], [1.0, 1.0]])
    loss, counts, mean, n, _ = ib.balance_loss(ln, [[1], [0]])
    assert counts.tolist() == [1, 1] and n == 2 and np.allclose(mean, [0.375, 0.625]) and np.isclose(loss, 1.0)
    loss, counts, mean, n, _ = ib.balance_loss(ln, [[1], [0]], [1, 0])
    assert counts.tolist() == [0, 1] and n == 1 and np.isclose(loss, 2 * 0.75)
    assert ib.balance_loss(ln, [[1], [0]], [0, 0])[0] == 0


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(3)
    T, E, k = 6, 5, 2
    logits = rng.standard_normal((T, E))
    logits[2, 3] = -np.inf
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)])
    mask = np.array([1, 1, 1, 0, 1, 1])
    _, counts, _, n, _ = ib.balance_loss(logits, ids, mask)
    d, _ = ib.balance_loss_backward(1.7, logits, counts, n, k, mask)
    for t in range(T):
        for e in range(E):
            def at(h):
                z = logits.copy()
                z[t, e] += h
                return 1.7 * ib.balance_loss(z, ids, mask)[0]
            # central differences of 1e-4 leave 1e-8 of the third derivative, and 1e-12 of rounding
            assert abs((at(1e-4) - at(-1e-4)) / 2e-4 - d[t, e]) < 1e-7


# ---------------------------------------------------------------------------
# what the compiler made
# ---------------------------------------------------------------------------
SOURCES = ("int8.hip", "int8_gemm.hip", "balance.hip")


def test_kernels_use_no_scratch(tmp_path):
    from test_build_resources import HAVE_HIPCC, _resources
    if not HAVE_HIPCC:
        pytest.skip("hipcc missing")
    for src in SOURCES:
        for name, r in _resources(src, tmp_path).items():
            assert r["scratch"] == 0 and r["spill"] == 0, (src, name, r)


def kernels_of(asm):
    """{name: its instructions and labels} of the kernels in an assembly listing."""
    out, name = {}, None
    for line in asm.split("\n"):
        line = line.split(";")[0].strip()
        m = re.match(r"(_ZN7moelora\w+):", line)
        if m:
            name = m.group(1)
            out[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name and line and (not line.startswith(".") or line.startswith(".LBB")):
            out[name].append(line)
    return out


def named(text):
    """Registers ("a" accumulators, "v") that operands name, as (kind, number)."""
    regs = set()
    for m in re.finditer(r"\b([av])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        lo, hi = (m.group(2), m.group(3)) if m.group(2) else (m.group(4), m.group(4))
        regs.update((m.group(1), i) for i in range(int(lo), int(hi) + 1))
    return regs


def early_uses(code):
    """Instructions that touch, over any path, a register that a matrix instruction wrote fewer
    than 18 wait states before, or matrix instructions that read one that the vector unit
    wrote fewer than 2 before."""
    labels = {line[:-1]: i for i, line in enumerate(code) if line.endswith(":")}
    found, before, work = [], {0: {}}, [0]
    while work:
        i = work.pop()
        state = dict(before[i])           # register: (its writer, wait states that are left)
        op, _, rest = code[i].partition(" ")
        regs, mfma, cost = named(rest), op.startswith("v_mfma"), 1
        if code[i].endswith(":"):
            cost = 0
        elif op == "s_nop":
            cost = int(rest, 0) + 1
        elif any(state.get(r, (mfma,))[0] != mfma for r in regs if mfma or state.get(r, (False,))[0]):
            found.append(code[i])
        state = {r: (w, n - cost) for r, (w, n) in state.items() if n > cost}
        if mfma:
            state.update({r: (True, 18) for r in named(rest.split(",")[0])})
        elif op.startswith("v_") and not op.startswith("v_cmp"):
            state.update({r: (False, 2) for r in named(rest.split(",")[0])})
        nexts = [] if op in ("s_endpgm", "s_branch") else [i + 1]
        if op == "s_branch" or op.startswith("s_cbranch"):
            nexts.append(labels[rest])
        for j in nexts:
            old = before.get(j)
            new = dict(old or {})
            for r, (w, n) in state.items():
                if r not in new or (w, n) > new[r]:
                    new[r] = (w, n)
            if old != new:
                before[j] = new
                work.append(j)
    return found


def test_early_uses_are_found():
    mul = "v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]"
    read = "v_accvgpr_read_b32 v9, a2"
    assert early_uses([mul, "s_nop 15", read, "s_endpgm"])
    assert not early_uses([mul, "s_nop 15", "s_nop 1", read, "s_endpgm"])
    assert early_uses(["v_mov_b32 v5, v9", "s_nop 0", mul, "s_endpgm"])
    assert not early_uses(["v_mov_b32 v5, v9", "s_nop 1", mul, "s_endpgm"])
    assert not early_uses([mul, mul, "v_mov_b32 v9, v0", "s_endpgm"])
    # over the loop's edge alone
    loop = ["s_branch .L1", ".L0:", mul, ".L1:", read, "s_cbranch_scc1 .L0", "s_endpgm"]
    assert early_uses(loop)
    assert not early_uses(loop[:3] + ["s_nop 15", "s_nop 1"] + loop[3:])


def test_results_of_matrix_instructions_are_waited_for(tmp_path):
    """The tile product's matrix instructions stand in assembly, where no one puts the waits in.
    No step of its loop moves an accumulator."""
    from test_build_resources import HAVE_HIPCC
    if not HAVE_HIPCC:
        pytest.skip("hipcc missing")
    out = tmp_path / "int8_gemm.s"
    subprocess.run([build.hipcc(), *build.common_flags(), "-S", "--cuda-device-only",
                    os.path.join(build.CSRC, "int8_gemm.hip"), "-o", str(out)], check=True)
    tiles = {n: c for n, c in kernels_of(out.read_text()).items() if "int8_tile" in n}
    assert len(tiles) == 3
    for name, code in tiles.items():
        assert not early_uses(code), (name, early_uses(code)[:3])
        at = [i for i, line in enumerate(code) if line.startswith("v_mfma")]
        back = [(i, code.index(line.split()[1] + ":")) for i, line in enumerate(code)
                if line.startswith(("s_branch", "s_cbranch"))]
        loops = [(j, i) for i, j in back if j < i and any(j < n < i for n in at)]
        assert loops
        for lo, hi in loops:
            moves = [line for line in code[lo:hi] if line.startswith("v_accvgpr")]
            assert not moves, (name, moves[:3])
