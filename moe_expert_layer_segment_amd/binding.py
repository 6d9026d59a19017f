"""ctypes binding of the gfx950 MoE-LoRA library (argument marshalling only).

Every step of the layer runs in the HIP kernels behind ``include/moe_lora.h``;
this module only checks tensor shapes / dtypes / devices, allocates outputs and
workspaces with PyTorch, and passes raw device pointers and the current HIP
stream.  If the shared library is missing it raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MOE_LORA_LIB") or os.path.join(_PKG, "lib", "libmoe_lora.so")
# the same library built with MOE_LORA_DEBUG (device-side precondition checks)
DEBUG_LIB_PATH = os.path.join(_PKG, "lib", "libmoe_lora_debug.so")

OK, ERR_INVALID, ERR_UNDERCOVER, ERR_UNSUPPORTED, ERR_HIP, ERR_WORKSPACE = 0, -1, -2, -3, -4, -5
DTYPE_F32, DTYPE_BF16, DTYPE_FP8_E4M3, DTYPE_U8, DTYPE_MX4 = 0, 1, 2, 3, 4
_FP8_TORCH = (torch.uint8, torch.float8_e4m3fn)   # one-byte e4m3 codes
FORWARD_STAGES = ("plan", "shrink_gate_up", "gate_up_gemm", "shrink_down", "down_gemm", "combine")

_c_i32p = ctypes.POINTER(ctypes.c_int32)


class ForwardArgs(ctypes.Structure):
    """Mirror of ``moe_lora_forward_args``."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("dtype", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
        ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("num_loras", ctypes.c_int32),
        ("max_rank", ctypes.c_int32), ("block_m", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p), ("topk_weights", ctypes.c_void_p),
        ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
        ("a_gate", ctypes.c_void_p), ("a_up", ctypes.c_void_p), ("b_gate", ctypes.c_void_p),
        ("b_up", ctypes.c_void_p), ("a_down", ctypes.c_void_p), ("b_down", ctypes.c_void_p),
        ("lora_ranks", ctypes.c_void_p), ("scaling", ctypes.c_void_p),
        ("sorted_pair_ids", ctypes.c_void_p), ("tile_expert", ctypes.c_void_p),
        ("tile_lora", ctypes.c_void_p), ("expert_tile_offsets", ctypes.c_void_p),
        ("num_rows_padded", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("y", ctypes.c_void_p), ("out_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("w_gate_up_scale", ctypes.c_void_p), ("w_down_scale", ctypes.c_void_p),
    ]


_LIB = None
_DEBUG_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        _LIB = _load(LIB_PATH)
    return _LIB


def debug_lib() -> ctypes.CDLL:
    """The MOE_LORA_DEBUG build of the library (same calls, same results; info
    and align also flag device-side precondition violations, read with
    ``moe_lora_debug_flags``)."""
    global _DEBUG_LIB
    if _DEBUG_LIB is None:
        _DEBUG_LIB = _load(DEBUG_LIB_PATH)
    return _DEBUG_LIB


def _load(path: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(
            f"MoE-LoRA HIP library not found at {path}; build it with "
            "`python -m moe_expert_layer_segment_amd.build` (no CPU fallback exists)")
    L = ctypes.CDLL(path)
    L.moe_lora_status_str.restype = ctypes.c_char_p
    L.moe_lora_status_str.argtypes = [ctypes.c_int]
    L.moe_lora_route.restype = ctypes.c_int
    L.moe_lora_route.argtypes = [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 4
    L.moe_lora_info.restype = ctypes.c_int
    L.moe_lora_info.argtypes = [ctypes.c_int32] * 4 + [ctypes.c_void_p] * 6
    L.moe_lora_align_capacity_rows.restype = ctypes.c_int64
    L.moe_lora_align_capacity_rows.argtypes = [ctypes.c_int32] * 5
    L.moe_lora_align_workspace_bytes.restype = ctypes.c_size_t
    L.moe_lora_align_workspace_bytes.argtypes = [ctypes.c_int32] * 5
    L.moe_lora_align.restype = ctypes.c_int
    L.moe_lora_align.argtypes = ([ctypes.c_int32] * 5 + [ctypes.c_void_p] * 9 +
                                 [ctypes.c_size_t, ctypes.c_void_p])
    L.moe_lora_align_pair_rows.restype = ctypes.c_int
    L.moe_lora_align_pair_rows.argtypes = ([ctypes.c_int32] * 5 + [ctypes.c_void_p] * 10 +
                                           [ctypes.c_size_t, ctypes.c_void_p])
    L.moe_lora_permute.restype = ctypes.c_int
    L.moe_lora_permute.argtypes = [ctypes.c_int32] * 4 + [ctypes.c_int64] + [ctypes.c_void_p] * 6
    L.moe_lora_permute_backward.restype = ctypes.c_int
    L.moe_lora_permute_backward.argtypes = ([ctypes.c_int32] * 5 + [ctypes.c_int64] +
                                            [ctypes.c_void_p] * 4)
    L.moe_lora_unpermute.restype = ctypes.c_int
    L.moe_lora_unpermute.argtypes = [ctypes.c_int32] * 5 + [ctypes.c_int64] + [ctypes.c_void_p] * 5
    L.moe_lora_unpermute_backward.restype = ctypes.c_int
    L.moe_lora_unpermute_backward.argtypes = ([ctypes.c_int32] * 5 + [ctypes.c_int64] +
                                              [ctypes.c_void_p] * 9)
    L.moe_lora_mx4_quantize.restype = ctypes.c_int
    L.moe_lora_mx4_quantize.argtypes = ([ctypes.c_int64] + [ctypes.c_int32] * 2 +
                                        [ctypes.c_void_p] * 5)
    L.moe_lora_mx4_dequantize.restype = ctypes.c_int
    L.moe_lora_mx4_dequantize.argtypes = ([ctypes.c_int64] + [ctypes.c_int32] * 2 +
                                          [ctypes.c_void_p] * 4)
    L.moe_lora_mx4_gemm.restype = ctypes.c_int
    L.moe_lora_mx4_gemm.argtypes = [ctypes.POINTER(Mx4GemmArgs), ctypes.c_void_p]
    L.moe_lora_forward_workspace_bytes.restype = ctypes.c_size_t
    L.moe_lora_forward_workspace_bytes.argtypes = [ctypes.POINTER(ForwardArgs)]
    L.moe_lora_forward.restype = ctypes.c_int
    L.moe_lora_forward.argtypes = [ctypes.POINTER(ForwardArgs), ctypes.c_void_p]
    L.moe_lora_forward_events.restype = ctypes.c_int
    L.moe_lora_forward_events.argtypes = [ctypes.POINTER(ForwardArgs), ctypes.c_void_p,
                                          ctypes.POINTER(ctypes.c_void_p)]
    L.moe_lora_dense_workspace_bytes.restype = ctypes.c_size_t
    L.moe_lora_dense_workspace_bytes.argtypes = [ctypes.POINTER(DenseArgs)]
    L.moe_lora_dense_forward.restype = ctypes.c_int
    L.moe_lora_dense_forward.argtypes = [ctypes.POINTER(DenseArgs), ctypes.c_void_p]
    L.moe_lora_dense_forward_events.restype = ctypes.c_int
    L.moe_lora_dense_forward_events.argtypes = [ctypes.POINTER(DenseArgs), ctypes.c_void_p,
                                                ctypes.POINTER(ctypes.c_void_p)]
    L.moe_lora_forward_noalloc.restype = ctypes.c_int
    L.moe_lora_forward_noalloc.argtypes = [ctypes.POINTER(ForwardArgs), ctypes.c_void_p]
    L.moe_lora_forward_noalloc_max_workspace_bytes.restype = ctypes.c_size_t
    L.moe_lora_forward_noalloc_max_workspace_bytes.argtypes = []
    L.moe_lora_debug_flags.restype = ctypes.c_int
    L.moe_lora_debug_flags.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int32,
                                       ctypes.c_void_p]
    return L


DEBUG_SEG_INDPTR, DEBUG_WEIGHT_INDEX, DEBUG_RANK, DEBUG_EXPERT_ID, DEBUG_MAPPING = 1, 2, 4, 8, 16


def debug_flags(clear: bool = True, library: Optional[ctypes.CDLL] = None) -> int:
    """The precondition flag word of a MOE_LORA_DEBUG build (after synchronising
    the current stream); ``clear`` resets it."""
    L = library or debug_lib()
    v = ctypes.c_uint32(0)
    _check(L.moe_lora_debug_flags(ctypes.byref(v), int(clear), _stream()), "moe_lora_debug_flags")
    return int(v.value)


class MoeLoraError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {lib().moe_lora_status_str(status).decode()} (status {status})")
        self.status = status


def _check(status: int, where: str):
    if status == ERR_UNDERCOVER:
        # the pages' unit test expects an AssertionError naming under-coverage
        raise AssertionError(f"{where}: launch under-covers tokens")
    if status != OK:
        raise MoeLoraError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t: torch.Tensor, name: str, dtype=None, device=None, numel=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} needs at least {numel} elements, has {t.numel()}")


# torch.cuda.current_stream builds a Stream object, which takes as long as a small kernel
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(where, device, call, *args):
    """call(*args, stream) with ``device`` as the current one, on its current stream."""
    index = device.index
    if index == torch.cuda.current_device():
        status = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, _raw_stream(index))
    if status != OK:
        _check(status, where)


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------
def moe_lora_route(logits: torch.Tensor, top_k: int, topk_ids: Optional[torch.Tensor] = None,
                   topk_weights: Optional[torch.Tensor] = None):
    """(topk_ids int32 [T, k], topk_weights fp32 [T, k]) from fp32 router logits [T, E]."""
    _need(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    if topk_weights is None:
        topk_weights = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    _need(topk_ids, "topk_ids", torch.int32, logits.device, T * top_k)
    _need(topk_weights, "topk_weights", torch.float32, logits.device, T * top_k)
    _check(lib().moe_lora_route(T, E, top_k, _ptr(logits), _ptr(topk_ids), _ptr(topk_weights),
                                _stream()), "moe_lora_route")
    return topk_ids, topk_weights


# ---------------------------------------------------------------------------
# info
# ---------------------------------------------------------------------------
def moe_lora_info(num_tokens: int, seg_indptr: torch.Tensor, lora_ranks: torch.Tensor,
                  weight_indices: torch.Tensor, adapter_enabled: Optional[torch.Tensor] = None,
                  token_lora_mapping: Optional[torch.Tensor] = None, max_len: int = 0):
    """Per-batch metadata; returns (adapter_enabled, token_lora_mapping[:num_tokens]).

    Argument order follows the pages' ``_compute_moe_lora_info``.  Preallocated
    outputs are written in place and returned as views of the same storage.
    Raises AssertionError when num_reqs * max_len < num_tokens.
    """
    dev = seg_indptr.device
    num_reqs = seg_indptr.numel() - 1
    num_loras = lora_ranks.numel()
    _need(seg_indptr, "seg_indptr", torch.int32)
    _need(lora_ranks, "lora_ranks", torch.int32, dev)
    _need(weight_indices, "weight_indices", torch.int32, dev, num_reqs)
    if adapter_enabled is None:
        adapter_enabled = torch.empty(num_loras, dtype=torch.int32, device=dev)
    if token_lora_mapping is None:
        token_lora_mapping = torch.empty(max(num_tokens, 1), dtype=torch.int32, device=dev)
    _need(adapter_enabled, "adapter_enabled", torch.int32, dev, num_loras)
    _need(token_lora_mapping, "token_lora_mapping", torch.int32, dev, num_tokens)
    st = lib().moe_lora_info(num_tokens, num_reqs, num_loras, int(max_len), _ptr(seg_indptr),
                             _ptr(weight_indices), _ptr(lora_ranks), _ptr(adapter_enabled),
                             _ptr(token_lora_mapping), _stream())
    _check(st, "moe_lora_info")
    return adapter_enabled, token_lora_mapping[:num_tokens]


compute_moe_lora_info = moe_lora_info


# ---------------------------------------------------------------------------
# align
# ---------------------------------------------------------------------------
def moe_lora_align_capacity_rows(num_tokens, top_k, num_experts, num_loras, block_m) -> int:
    v = lib().moe_lora_align_capacity_rows(num_tokens, top_k, num_experts, num_loras, block_m)
    if v < 0:
        raise MoeLoraError(ERR_INVALID, "moe_lora_align_capacity_rows")
    return int(v)


def moe_lora_align_workspace_bytes(num_tokens, top_k, num_experts, num_loras, block_m) -> int:
    return int(lib().moe_lora_align_workspace_bytes(num_tokens, top_k, num_experts, num_loras,
                                                    block_m))


def moe_lora_align(topk_ids: torch.Tensor, token_lora_mapping: torch.Tensor,
                   adapter_enabled: Optional[torch.Tensor], num_experts: int, num_loras: int,
                   block_m: int = 16, out: Optional[Dict[str, torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None,
                   pair_rows: bool = False) -> Dict[str, torch.Tensor]:
    """Bucket (token, expert) pairs by (expert, adapter); returns the align outputs.

    ``pair_rows``: also write ``pair_rows`` (int32 [T * k], the row of each pair or
    -1), which moe_lora_permute and moe_lora_unpermute need.  None stay from a batch before:
    where ``out`` holds a buffer for them they are written unasked, or the buffer leaves it
    if it is too small.  Buffers in ``out`` may be larger than this batch needs;
    ``num_pairs`` in the result says how many pairs it has."""
    dev = topk_ids.device
    T, k = topk_ids.shape
    _need(topk_ids, "topk_ids", torch.int32)
    _need(token_lora_mapping, "token_lora_mapping", torch.int32, dev, T)
    if num_loras > 0:
        _need(adapter_enabled, "adapter_enabled", torch.int32, dev, num_loras)
    cap = moe_lora_align_capacity_rows(T, k, num_experts, num_loras, block_m)
    if out is None:
        out = dict(
            sorted_pair_ids=torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
            tile_expert=torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev),
            tile_lora=torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev),
            expert_tile_offsets=torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
            num_rows_padded=torch.empty(1, dtype=torch.int32, device=dev))
    held = out.get("pair_rows")
    if held is not None and not pair_rows:
        pair_rows = held.numel() >= T * k
        if not pair_rows:
            del out["pair_rows"]
    if pair_rows:
        if held is None:
            out["pair_rows"] = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
        _need(out["pair_rows"], "pair_rows", torch.int32, dev, T * k)
    for name, n in (("sorted_pair_ids", cap), ("tile_expert", cap // block_m),
                    ("tile_lora", cap // block_m), ("expert_tile_offsets", num_experts + 1),
                    ("num_rows_padded", 1)):
        _need(out[name], name, torch.int32, dev, n)
    wsb = moe_lora_align_workspace_bytes(T, k, num_experts, num_loras, block_m)
    if workspace is None:
        workspace = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev, wsb)
    args = [T, k, num_experts, num_loras, block_m, _ptr(topk_ids), _ptr(token_lora_mapping),
            _ptr(adapter_enabled) if num_loras > 0 else None, _ptr(out["sorted_pair_ids"]),
            _ptr(out["tile_expert"]), _ptr(out["tile_lora"]), _ptr(out["expert_tile_offsets"]),
            _ptr(out["num_rows_padded"])]
    if pair_rows:
        _launch("moe_lora_align", dev, lib().moe_lora_align_pair_rows, *args, _ptr(out["pair_rows"]),
                _ptr(workspace), workspace.numel())
    else:
        _launch("moe_lora_align", dev, lib().moe_lora_align, *args, _ptr(workspace), workspace.numel())
    out["capacity"] = cap
    out["block_m"] = block_m
    out["num_pairs"] = T * k
    return out


# ---------------------------------------------------------------------------
# forward
# ---------------------------------------------------------------------------
_POOLS = ("a_gate", "a_up", "b_gate", "b_up", "a_down", "b_down")


def _forward_args(x, topk_weights, w_gate_up, w_down, align_out, lora_ranks, scaling, pools,
                  top_k, y, workspace, out_dtype=None, w_scales=None) -> ForwardArgs:
    T, H = x.shape
    E, twoI, H2 = w_gate_up.shape
    I = twoI // 2
    if x.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif x.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError(f"unsupported dtype {x.dtype}")
    dev = x.device
    _need(x, "x", x.dtype)
    fp8 = w_gate_up.dtype in _FP8_TORCH
    wdt = w_gate_up.dtype if fp8 else x.dtype
    _need(w_gate_up, "w_gate_up", wdt, dev)
    _need(w_down, "w_down", wdt, dev)
    if H2 != H or tuple(w_down.shape) != (E, H, I):
        raise ValueError("weight shapes do not match x / each other")
    if fp8:
        if x.dtype != torch.bfloat16:
            raise TypeError("fp8 expert weights need bf16 activations")
        if w_scales is None:
            raise ValueError("fp8 expert weights need their block scales (w_scales)")
        sgu, sd = w_scales
        _need(sgu, "w_gate_up_scale", torch.float32, dev)
        _need(sd, "w_down_scale", torch.float32, dev)
        if tuple(sgu.shape) != (E, 2 * I // 128, H // 128) or tuple(sd.shape) != (E, H // 128, I // 128):
            raise ValueError("block scales must be [E, 2I/128, H/128] and [E, H/128, I/128]")
    _need(topk_weights, "topk_weights", torch.float32, dev, T * top_k)
    L, R = 0, 0
    if pools is not None:
        L, E2, R, _ = pools["a_gate"].shape
        if E2 != E:
            raise ValueError("pool expert axis does not match the weights")
        shapes = dict(a_gate=(L, E, R, H), a_up=(L, E, R, H), b_gate=(L, E, R, I),
                      b_up=(L, E, R, I), a_down=(L, E, R, I), b_down=(L, E, R, H))
        for n in _POOLS:
            _need(pools[n], n, x.dtype, dev)
            if tuple(pools[n].shape) != shapes[n]:
                raise ValueError(f"{n} must have shape {shapes[n]}, got {tuple(pools[n].shape)}")
        _need(lora_ranks, "lora_ranks", torch.int32, dev, L)
        _need(scaling, "scaling", torch.float32, dev, L)
    a = ForwardArgs()
    a.struct_size = ctypes.sizeof(ForwardArgs)
    a.dtype = dt
    out_dt = x.dtype if out_dtype is None else out_dtype
    if out_dt == torch.float32:
        a.out_dtype = DTYPE_F32
    elif out_dt == x.dtype:
        a.out_dtype = dt
    else:
        raise TypeError(f"unsupported output dtype {out_dt}")
    a.num_tokens, a.hidden, a.inter, a.num_experts, a.top_k = T, H, I, E, top_k
    a.num_loras, a.max_rank, a.block_m = L, R, int(align_out["block_m"])
    a.x, a.topk_weights = x.data_ptr(), topk_weights.data_ptr()
    a.w_gate_up, a.w_down = w_gate_up.data_ptr(), w_down.data_ptr()
    if fp8:
        a.weight_dtype = DTYPE_FP8_E4M3
        a.w_gate_up_scale, a.w_down_scale = w_scales[0].data_ptr(), w_scales[1].data_ptr()
    if pools is not None:
        for n in _POOLS:
            setattr(a, n, pools[n].data_ptr())
        a.lora_ranks, a.scaling = lora_ranks.data_ptr(), scaling.data_ptr()
    for n in ("sorted_pair_ids", "tile_expert", "tile_lora", "expert_tile_offsets",
              "num_rows_padded"):
        _need(align_out[n], n, torch.int32, dev)
        setattr(a, n, align_out[n].data_ptr())
    if y is not None:
        _need(y, "y", out_dt, dev, T * H)
        a.y = y.data_ptr()
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return a


def moe_lora_forward_workspace_bytes(x, topk_weights, w_gate_up, w_down, align_out, top_k,
                                     lora_ranks=None, scaling=None, pools=None,
                                     w_scales=None) -> int:
    a = _forward_args(x, topk_weights, w_gate_up, w_down, align_out, lora_ranks, scaling, pools,
                      top_k, None, None, w_scales=w_scales)
    n = int(lib().moe_lora_forward_workspace_bytes(ctypes.byref(a)))
    if n == 0:
        raise MoeLoraError(ERR_INVALID, "moe_lora_forward_workspace_bytes")
    return n


def moe_lora_forward(x: torch.Tensor, topk_weights: torch.Tensor, w_gate_up: torch.Tensor,
                     w_down: torch.Tensor, align_out: Dict[str, torch.Tensor], top_k: int,
                     lora_ranks: Optional[torch.Tensor] = None,
                     scaling: Optional[torch.Tensor] = None,
                     pools: Optional[Dict[str, torch.Tensor]] = None,
                     y: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     events=None, out_dtype=None, w_scales=None) -> torch.Tensor:
    """The MoE-LoRA layer: returns y [T, H] (written into ``y`` if given).

    fp8 expert weights: ``w_gate_up`` / ``w_down`` as uint8 or float8_e4m3fn
    e4m3 codes and ``w_scales`` = (gate_up scales [E, 2I/128, H/128], down
    scales [E, H/128, I/128]), float32.

    ``events``: optional sequence of 2 * len(FORWARD_STAGES) raw hipEvent_t
    handles recorded around each kernel stage (measurement only).
    """
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype if out_dtype is None else out_dtype,
                        device=x.device)
    if workspace is None:
        n = moe_lora_forward_workspace_bytes(x, topk_weights, w_gate_up, w_down, align_out, top_k,
                                             lora_ranks, scaling, pools, w_scales)
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    a = _forward_args(x, topk_weights, w_gate_up, w_down, align_out, lora_ranks, scaling, pools,
                      top_k, y, workspace, out_dtype, w_scales)
    if events is None:
        _check(lib().moe_lora_forward(ctypes.byref(a), _stream()), "moe_lora_forward")
    else:
        if len(events) != 2 * len(FORWARD_STAGES):
            raise ValueError("events needs one pair per forward stage")
        arr = (ctypes.c_void_p * len(events))(*events)
        _check(lib().moe_lora_forward_events(ctypes.byref(a), _stream(), arr),
               "moe_lora_forward_events")
    return y


def moe_lora_forward_noalloc(x: torch.Tensor, topk_weights: torch.Tensor, w_gate_up: torch.Tensor,
                             w_down: torch.Tensor, align_out: Dict[str, torch.Tensor], top_k: int,
                             lora_ranks: Optional[torch.Tensor] = None,
                             scaling: Optional[torch.Tensor] = None,
                             pools: Optional[Dict[str, torch.Tensor]] = None,
                             y: Optional[torch.Tensor] = None, out_dtype=None,
                             w_scales=None) -> torch.Tensor:
    """moe_lora_forward without a caller workspace: the library's static
    per-device scratch serves instead (problems up to
    ``moe_lora_forward_noalloc_max_workspace_bytes()``; calls on one device must
    not overlap).  Only ``y`` is allocated here, and only when not given."""
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype if out_dtype is None else out_dtype,
                        device=x.device)
    a = _forward_args(x, topk_weights, w_gate_up, w_down, align_out, lora_ranks, scaling, pools,
                      top_k, y, None, out_dtype, w_scales)
    _check(lib().moe_lora_forward_noalloc(ctypes.byref(a), _stream()), "moe_lora_forward_noalloc")
    return y


def moe_lora_forward_noalloc_max_workspace_bytes() -> int:
    return int(lib().moe_lora_forward_noalloc_max_workspace_bytes())


def run_layer(inputs: dict, block_m: int = 16, with_lora: bool = True,
              out_dtype=None) -> torch.Tensor:
    """info -> align -> forward on a dict from ``workloads.generate``."""
    T = inputs["x"].shape[0]
    k = inputs["topk_ids"].shape[1]
    E = inputs["w_gate_up"].shape[0]
    L = inputs["lora_ranks"].numel() if with_lora and "a_gate" in inputs else 0
    ranks = inputs["lora_ranks"]
    en, mp = moe_lora_info(T, inputs["seg_indptr"], ranks, inputs["weight_indices"],
                           max_len=inputs["meta"]["max_seg_len"])
    al = moe_lora_align(inputs["topk_ids"], mp, en if L > 0 else None, E, L, block_m)
    pools = {n: inputs[n] for n in _POOLS} if L > 0 else None
    ws = ((inputs["w_gate_up_scale"], inputs["w_down_scale"])
          if "w_gate_up_scale" in inputs else None)
    return moe_lora_forward(inputs["x"], inputs["topk_weights"], inputs["w_gate_up"],
                            inputs["w_down"], al, k, ranks if L > 0 else None,
                            inputs["scaling"] if L > 0 else None, pools, out_dtype=out_dtype,
                            w_scales=ws)


# ---------------------------------------------------------------------------
# dense projection with a two-slice LoRA output
# ---------------------------------------------------------------------------
DENSE_STAGES = ("plan", "shrink", "gemm", "combine")


class DenseArgs(ctypes.Structure):
    """Mirror of ``moe_lora_dense_args``."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("dtype", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("out0", ctypes.c_int32),
        ("out1", ctypes.c_int32), ("num_loras", ctypes.c_int32), ("max_rank", ctypes.c_int32),
        ("block_m", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("w", ctypes.c_void_p),
        ("a0", ctypes.c_void_p), ("a1", ctypes.c_void_p), ("b0", ctypes.c_void_p),
        ("b1", ctypes.c_void_p),
        ("lora_ranks", ctypes.c_void_p), ("scaling", ctypes.c_void_p),
        ("sorted_pair_ids", ctypes.c_void_p), ("tile_expert", ctypes.c_void_p),
        ("tile_lora", ctypes.c_void_p), ("expert_tile_offsets", ctypes.c_void_p),
        ("num_rows_padded", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("y", ctypes.c_void_p), ("out_dtype", ctypes.c_int32),
    ]


def _dense_args(x, w, out0, align_out, lora_ranks, scaling, pools, y, workspace,
                out_dtype=None) -> DenseArgs:
    T, H = x.shape
    N, H2 = w.shape
    if H2 != H or not (0 < out0 <= N):
        raise ValueError("w must be [out0 + out1, H] with 0 < out0 <= its rows")
    if x.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif x.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError(f"unsupported dtype {x.dtype}")
    dev = x.device
    _need(x, "x", x.dtype)
    _need(w, "w", x.dtype, dev)
    out1 = N - out0
    L, R = 0, 0
    if pools is not None:
        L, R, _ = pools["a0"].shape
        shapes = dict(a0=(L, R, H), a1=(L, R, H), b0=(L, R, out0), b1=(L, R, out1))
        for n in ("a0", "b0") + (("a1", "b1") if out1 > 0 else ()):
            _need(pools[n], n, x.dtype, dev)
            if tuple(pools[n].shape) != shapes[n]:
                raise ValueError(f"{n} must have shape {shapes[n]}, got {tuple(pools[n].shape)}")
        _need(lora_ranks, "lora_ranks", torch.int32, dev, L)
        _need(scaling, "scaling", torch.float32, dev, L)
    a = DenseArgs()
    a.struct_size = ctypes.sizeof(DenseArgs)
    a.dtype = dt
    out_dt = x.dtype if out_dtype is None else out_dtype
    if out_dt == torch.float32:
        a.out_dtype = DTYPE_F32
    elif out_dt == x.dtype:
        a.out_dtype = dt
    else:
        raise TypeError(f"unsupported output dtype {out_dt}")
    a.num_tokens, a.hidden, a.out0, a.out1 = T, H, out0, out1
    a.num_loras, a.max_rank, a.block_m = L, R, int(align_out["block_m"])
    a.x, a.w = x.data_ptr(), w.data_ptr()
    if pools is not None:
        a.a0, a.b0 = pools["a0"].data_ptr(), pools["b0"].data_ptr()
        if out1 > 0:
            a.a1, a.b1 = pools["a1"].data_ptr(), pools["b1"].data_ptr()
        a.lora_ranks, a.scaling = lora_ranks.data_ptr(), scaling.data_ptr()
    for n in ("sorted_pair_ids", "tile_expert", "tile_lora", "expert_tile_offsets",
              "num_rows_padded"):
        _need(align_out[n], n, torch.int32, dev)
        setattr(a, n, align_out[n].data_ptr())
    if y is not None:
        _need(y, "y", out_dt, dev, T * N)
        a.y = y.data_ptr()
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return a


def moe_lora_dense_workspace_bytes(x, w, out0, align_out, lora_ranks=None, scaling=None,
                                   pools=None) -> int:
    a = _dense_args(x, w, out0, align_out, lora_ranks, scaling, pools, None, None)
    n = int(lib().moe_lora_dense_workspace_bytes(ctypes.byref(a)))
    if n == 0:
        raise MoeLoraError(ERR_INVALID, "moe_lora_dense_workspace_bytes")
    return n


def moe_lora_dense_forward(x: torch.Tensor, w: torch.Tensor, out0: int,
                           align_out: Dict[str, torch.Tensor],
                           lora_ranks: Optional[torch.Tensor] = None,
                           scaling: Optional[torch.Tensor] = None,
                           pools: Optional[Dict[str, torch.Tensor]] = None,
                           y: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           events=None, out_dtype=None) -> torch.Tensor:
    """Dense projection with per-request LoRA and two output slices: y [T, N]
    (``pools``: a0, a1 [L, R, H], b0 [L, R, out0], b1 [L, R, N - out0]).
    ``align_out`` comes from moe_lora_align with one expert and top_k = 1."""
    T = x.shape[0]
    N = w.shape[0]
    if y is None:
        y = torch.empty((T, N), dtype=x.dtype if out_dtype is None else out_dtype, device=x.device)
    if workspace is None:
        n = moe_lora_dense_workspace_bytes(x, w, out0, align_out, lora_ranks, scaling, pools)
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    a = _dense_args(x, w, out0, align_out, lora_ranks, scaling, pools, y, workspace, out_dtype)
    if events is None:
        _check(lib().moe_lora_dense_forward(ctypes.byref(a), _stream()), "moe_lora_dense_forward")
    else:
        if len(events) != 2 * len(DENSE_STAGES):
            raise ValueError("events needs one pair per dense stage")
        arr = (ctypes.c_void_p * len(events))(*events)
        _check(lib().moe_lora_dense_forward_events(ctypes.byref(a), _stream(), arr),
               "moe_lora_dense_forward_events")
    return y


def run_dense(inputs: dict, out0: int, block_m: int = 16, with_lora: bool = True,
              out_dtype=None) -> torch.Tensor:
    """info -> align (one expert, top_k = 1) -> dense forward on a dict from
    ``workloads.generate_dense``."""
    T = inputs["x"].shape[0]
    L = inputs["lora_ranks"].numel() if with_lora and "a0" in inputs else 0
    ranks = inputs["lora_ranks"]
    en, mp = moe_lora_info(T, inputs["seg_indptr"], ranks, inputs["weight_indices"],
                           max_len=inputs["meta"]["max_seg_len"])
    al = moe_lora_align(inputs["topk_ids"], mp, en if L > 0 else None, 1, L, block_m)
    pools = {n: inputs[n] for n in ("a0", "a1", "b0", "b1")} if L > 0 else None
    return moe_lora_dense_forward(inputs["x"], inputs["w"], out0, al, ranks if L > 0 else None,
                                  inputs["scaling"] if L > 0 else None, pools,
                                  out_dtype=out_dtype)


# ---------------------------------------------------------------------------
# rows in expert order
# ---------------------------------------------------------------------------
_ROW_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _row_dtype(t, name, also=()):
    dtype = t if isinstance(t, torch.dtype) else t.dtype
    if dtype in _ROW_DTYPES:
        return _ROW_DTYPES[dtype]
    if dtype in also:
        return DTYPE_U8
    raise TypeError(f"unsupported dtype of {name}: {dtype}")


def _rows_layout(align_out, top_k, dev, num_rows=None):
    """(tokens, rows of the layout) after checking its arrays."""
    if "pair_rows" not in align_out:
        raise ValueError("the layout has no pair_rows (moe_lora_align(..., pair_rows=True))")
    pr, pairs, cap = align_out["pair_rows"], align_out.get("num_pairs"), int(align_out["capacity"])
    _need(pr, "pair_rows", torch.int32, dev)
    # pair_rows may be a buffer of more than the batch's pairs, or those of its first tokens
    held = pr.numel()
    if pairs is None or held < pairs:
        pairs = held
    _need(align_out["sorted_pair_ids"], "sorted_pair_ids", torch.int32, dev, cap)
    _need(align_out["num_rows_padded"], "num_rows_padded", torch.int32, dev, 1)
    if top_k <= 0 or (cap > 0 and pairs % top_k):
        raise ValueError("pair_rows is not [T, top_k]")
    if num_rows is not None and num_rows != cap:
        raise ValueError(f"the layout has {cap} rows, got {num_rows}")
    return (pairs // top_k if cap > 0 else 0), cap


def _layout_at(align_out):
    """Addresses of sorted_pair_ids, pair_rows and num_rows_padded."""
    return (align_out["sorted_pair_ids"].data_ptr(), align_out["pair_rows"].data_ptr(),
            align_out["num_rows_padded"].data_ptr())


def _apart(out, *inputs):
    """Outputs must not share memory with inputs; returns the output's first address and the
    one behind it."""
    lo = out.data_ptr()
    hi = lo + out.nbytes
    for t in inputs:
        if t is not None:
            p = t.data_ptr()
            if lo < p + t.nbytes and p < hi:
                raise ValueError("an output overlaps an input")
    return lo, hi


def _apart_from_layout(span, at, cap, pairs):
    """The same of an output's addresses and the arrays of the layout, at _layout_at."""
    lo, hi = span
    ids, pair_rows, used = at
    if (lo < ids + 4 * cap and ids < hi) or (lo < pair_rows + 4 * pairs and pair_rows < hi) or \
            (lo < used + 4 and used < hi):
        raise ValueError("an output overlaps the layout")


def _requires_grad(where):
    """For a call with an input that requires a gradient: autograd does not see these
    calls, and where it is on, the call is refused rather than the gradient lost."""
    if torch.is_grad_enabled():
        raise ValueError(f"{where} is not recorded by autograd and an input requires a gradient: "
                         "call it under torch.no_grad() or in a torch.autograd.Function")


def _matrix(t, name, dev=None):
    _need(t, name, None, dev)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def moe_lora_permute(x: torch.Tensor, align_out: Dict[str, torch.Tensor], top_k: int,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of x [T, H] copied to expert order: rows [capacity, H] of x's dtype
    (float32, bfloat16, or uint8 for MX4 codes and scales).

    Padding rows before ``num_rows_padded`` are zero; rows behind it are left as
    they are in ``out`` (undefined when it is not given).  ``align_out`` comes from
    moe_lora_align with ``pair_rows=True``.

    Like all calls on rows it is for torch.no_grad() or the forward and backward of a
    torch.autograd.Function: its gradient is moe_lora_permute_backward, and an x that
    requires a gradient is refused where autograd is on."""
    _matrix(x, "x")
    if x.requires_grad:
        _requires_grad("moe_lora_permute")
    dt = _row_dtype(x, "x", (torch.uint8,))
    T, cap = _rows_layout(align_out, top_k, x.device)
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, the layout {T} tokens")
    H, at = x.shape[1], _layout_at(align_out)
    if out is None:
        out = torch.empty((cap, H), dtype=x.dtype, device=x.device)
    else:
        _need(out, "out", x.dtype, x.device)
        if out.shape != (cap, H):
            raise ValueError(f"out must be {(cap, H)}, got {tuple(out.shape)}")
        _apart_from_layout(_apart(out, x), at, cap, T * top_k)
    _launch("moe_lora_permute", x.device, lib().moe_lora_permute, T, top_k, H, dt, cap, _at(x), *at,
            _at(out))
    return out


def moe_lora_permute_backward(d_rows: torch.Tensor, align_out: Dict[str, torch.Tensor], top_k: int,
                              dx: Optional[torch.Tensor] = None, out_dtype=None) -> torch.Tensor:
    """Gradient of moe_lora_permute: dx [T, H], the sum of each token's rows of
    ``d_rows`` (fp32 sums; ``out_dtype`` defaults to the rows' dtype)."""
    _matrix(d_rows, "d_rows")
    if d_rows.requires_grad:
        _requires_grad("moe_lora_permute_backward")
    T, cap = _rows_layout(align_out, top_k, d_rows.device, d_rows.shape[0])
    H = d_rows.shape[1]
    if dx is None:
        dx = torch.empty((T, H), dtype=out_dtype or d_rows.dtype, device=d_rows.device)
    else:
        _token_out(dx, "dx", T, H, out_dtype, d_rows)
        _apart_from_layout(_apart(dx, d_rows), _layout_at(align_out), cap, T * top_k)
    _launch("moe_lora_permute_backward", d_rows.device, lib().moe_lora_permute_backward, T, top_k, H,
            _row_dtype(d_rows, "d_rows"), _row_dtype(dx, "dx"), cap, _at(d_rows),
            _at(align_out["pair_rows"]), _at(dx))
    return dx


def _token_out(t, name, T, H, out_dtype, rows):
    _need(t, name, out_dtype, rows.device)
    if t.shape != (T, H):
        raise ValueError(f"{name} must be {(T, H)}, got {tuple(t.shape)}")


def _pair_weights(w, T, top_k, dev, name="topk_weights"):
    _need(w, name, torch.float32, dev)
    if w.numel() != T * top_k:
        raise ValueError(f"{name} must be [{T}, {top_k}], got {tuple(w.shape)}")


def moe_lora_unpermute(rows: torch.Tensor, align_out: Dict[str, torch.Tensor], top_k: int,
                       topk_weights: Optional[torch.Tensor] = None,
                       y: Optional[torch.Tensor] = None, out_dtype=None) -> torch.Tensor:
    """y [T, H] = the sum over a token's top_k pairs of weight times row (fp32,
    in pair order, rounded once; no weights: ones).  Pairs without a row take no
    part.  ``out_dtype`` defaults to the rows' dtype.  The gradients are those of
    moe_lora_unpermute_backward; rows or weights that require one are refused where
    autograd is on."""
    _matrix(rows, "rows")
    T, cap = _rows_layout(align_out, top_k, rows.device, rows.shape[0])
    H = rows.shape[1]
    if topk_weights is not None:
        _pair_weights(topk_weights, T, top_k, rows.device)
    if rows.requires_grad or (topk_weights is not None and topk_weights.requires_grad):
        _requires_grad("moe_lora_unpermute")
    if y is None:
        y = torch.empty((T, H), dtype=out_dtype or rows.dtype, device=rows.device)
    else:
        _token_out(y, "y", T, H, out_dtype, rows)
        _apart_from_layout(_apart(y, rows, topk_weights), _layout_at(align_out), cap, T * top_k)
    _launch("moe_lora_unpermute", rows.device, lib().moe_lora_unpermute, T, top_k, H,
            _row_dtype(rows, "rows"), _row_dtype(y, "y"), cap, _at(rows), _at(align_out["pair_rows"]),
            _at(topk_weights), _at(y))
    return y


def moe_lora_unpermute_backward(dy: torch.Tensor, rows: Optional[torch.Tensor],
                                align_out: Dict[str, torch.Tensor], top_k: int,
                                topk_weights: Optional[torch.Tensor] = None,
                                d_rows: Optional[torch.Tensor] = None,
                                d_weights: Optional[torch.Tensor] = None,
                                rows_dtype=None):
    """Gradients of moe_lora_unpermute: (d_rows [capacity, H], d_weights [T, top_k]).

    ``rows`` are the forward's rows, needed for d_weights; with ``rows=None`` (or
    without weights) d_weights is None, and d_rows takes ``rows_dtype`` (default
    dy's).  Padding rows of d_rows are zero, rows behind ``num_rows_padded`` are
    left as they are."""
    _matrix(dy, "dy")
    dev = dy.device
    T, cap = _rows_layout(align_out, top_k, dev)
    H = dy.shape[1]
    if dy.shape[0] != T:
        raise ValueError(f"dy has {dy.shape[0]} rows, the layout {T} tokens")
    if rows is not None:
        _need(rows, "rows", rows_dtype, dev)
        if rows.shape != (cap, H):
            raise ValueError(f"rows must be {(cap, H)}, got {tuple(rows.shape)}")
    if topk_weights is not None:
        _pair_weights(topk_weights, T, top_k, dev)
    for t in (dy, rows, topk_weights):
        if t is not None and t.requires_grad:
            _requires_grad("moe_lora_unpermute_backward")
    dt = rows.dtype if rows is not None else rows_dtype or dy.dtype
    if d_rows is None:
        d_rows = torch.empty((cap, H), dtype=dt, device=dev)
    _need(d_rows, "d_rows", dt, dev)
    if d_rows.shape != (cap, H):
        raise ValueError(f"d_rows must be {(cap, H)}, got {tuple(d_rows.shape)}")
    at = _layout_at(align_out)
    _apart_from_layout(_apart(d_rows, dy, rows, topk_weights), at, cap, T * top_k)
    if rows is None or topk_weights is None:
        if d_weights is not None:
            raise ValueError("d_weights needs rows and topk_weights")
    elif d_weights is None:
        d_weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    if d_weights is not None:
        _pair_weights(d_weights, T, top_k, dev, "d_weights")
        _apart_from_layout(_apart(d_weights, dy, rows, topk_weights, d_rows), at, cap, T * top_k)
    _launch("moe_lora_unpermute_backward", dev, lib().moe_lora_unpermute_backward, T, top_k, H,
            _row_dtype(dt, "rows"), _row_dtype(dy, "dy"), cap, _at(dy), _at(rows),
            *at, _at(topk_weights), _at(d_rows), _at(d_weights))
    return d_rows, d_weights


# ---------------------------------------------------------------------------
# MX4: 4-bit values in blocks of 32 under a power-of-two scale
# ---------------------------------------------------------------------------
class Mx4GemmArgs(ctypes.Structure):
    """Mirror of ``moe_lora_mx4_gemm_args``."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("x_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("num_rows", ctypes.c_int64),
        ("out_features", ctypes.c_int32), ("in_features", ctypes.c_int32),
        ("num_experts", ctypes.c_int32), ("block_m", ctypes.c_int32),
        ("silu_mul", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("x_scale", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("w_scale", ctypes.c_void_p),
        ("tile_expert", ctypes.c_void_p), ("sorted_pair_ids", ctypes.c_void_p),
        ("num_pairs", ctypes.c_int32), ("out", ctypes.c_void_p),
    ]


def _mx4_pair(codes, scales, name, dev=None):
    """Checks codes [.., K / 2] and scales [.., K / 32]; returns K."""
    _need(codes, f"{name} codes", torch.uint8, dev)
    _need(scales, f"{name} scales", torch.uint8, codes.device)
    if codes.dim() < 1 or codes.shape[-1] % 16 or \
            scales.shape != (*codes.shape[:-1], codes.shape[-1] // 16):
        raise ValueError(f"{name} must be codes [.., K/2] and scales [.., K/32], got "
                         f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    return 2 * codes.shape[-1]


def moe_lora_mx4_quantize(x: torch.Tensor, num_rows_used: Optional[torch.Tensor] = None,
                          codes: Optional[torch.Tensor] = None,
                          scales: Optional[torch.Tensor] = None):
    """(codes uint8 [.., K/2], scales uint8 [.., K/32]) of x [.., K], K a multiple of
    32, float32 or bfloat16.

    ``num_rows_used``: device int32 [1]; rows of x (all leading axes together) from
    it on are skipped, their outputs left as they are (``num_rows_padded`` of
    moe_lora_align)."""
    _need(x, "x")
    dt = _row_dtype(x, "x")
    K = x.shape[-1] if x.dim() else 0
    if K <= 0 or K % 32:
        raise ValueError("the last axis of x must be a multiple of 32")
    lead, dev = tuple(x.shape[:-1]), x.device
    if num_rows_used is not None:
        _need(num_rows_used, "num_rows_used", torch.int32, dev, 1)
    given = codes is not None or scales is not None
    if codes is None:
        codes = torch.empty((*lead, K // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((*lead, K // 32), dtype=torch.uint8, device=dev)
    if given:
        _mx4_pair(codes, scales, "the output", dev)
        if codes.shape != (*lead, K // 2):
            raise ValueError(f"codes must be {(*lead, K // 2)}, got {tuple(codes.shape)}")
        _apart(codes, x, scales, num_rows_used)
        _apart(scales, x, num_rows_used)
    _launch("moe_lora_mx4_quantize", dev, lib().moe_lora_mx4_quantize, x.numel() // K, K, dt, _at(x),
            _at(num_rows_used), _at(codes), _at(scales))
    return codes, scales


def moe_lora_mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor,
                            out: Optional[torch.Tensor] = None, out_dtype=None) -> torch.Tensor:
    """The values [.., K] that MX4 codes and scales stand for (bfloat16 unless
    ``out_dtype`` or ``out`` says float32)."""
    K = _mx4_pair(codes, scales, "x")
    shape = (*codes.shape[:-1], K)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or torch.bfloat16, device=codes.device)
    else:
        _need(out, "out", out_dtype, codes.device)
        if out.shape != shape:
            raise ValueError(f"out must be {shape}, got {tuple(out.shape)}")
        _apart(out, codes, scales)
    if K == 0:
        return out
    _launch("moe_lora_mx4_dequantize", codes.device, lib().moe_lora_mx4_dequantize, out.numel() // K, K,
            _row_dtype(out, "out"), _at(codes), _at(scales), _at(out))
    return out


def moe_lora_mx4_gemm(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                      x_scales: Optional[torch.Tensor] = None,
                      align_out: Optional[Dict[str, torch.Tensor]] = None, silu_mul: bool = False,
                      out: Optional[torch.Tensor] = None, out_dtype=None) -> torch.Tensor:
    """x W^T with MX4 weights; ``silu_mul``: SiLU(gate) * up of the two halves of the
    output columns.

    ``align_out`` None: w_codes [N, K/2], w_scales [N, K/32], x [M, K] of any M.
    Otherwise w_codes [E, N, K/2], w_scales [E, N, K/32] and x [capacity, K] in
    expert order (moe_lora_permute); rows behind the last used tile are left as they
    are in ``out`` (undefined when it is not given).  With ``pair_rows`` in align_out
    padding rows get zeros, whatever x and the weights hold.
    x: bfloat16, or MX4 codes [M, K/2] with ``x_scales`` [M, K/32].  ``out`` /
    ``out_dtype``: bfloat16 (the default) or float32.  There is no gradient: an x that
    requires one is refused where autograd is on."""
    K = _mx4_pair(w_codes, w_scales, "w")
    dev = w_codes.device
    if w_codes.dim() != (2 if align_out is None else 3):
        raise ValueError("w_codes must be [N, K/2], or [E, N, K/2] with align_out")
    E, N = (1 if align_out is None else w_codes.shape[0]), w_codes.shape[-2]
    if x_scales is None:
        _need(x, "x", torch.bfloat16, dev)
        if x.requires_grad:
            _requires_grad("moe_lora_mx4_gemm")
        xk = x.shape[-1] if x.dim() == 2 else -1
    else:
        xk = _mx4_pair(x, x_scales, "x", dev) if x.dim() == 2 else -1
    if x.dim() != 2 or xk != K:
        raise ValueError(f"x {tuple(x.shape)} does not match weights of {K} columns")
    M, a, layout = x.shape[0], Mx4GemmArgs(), ()
    if align_out is not None:
        a.block_m = int(align_out["block_m"])
        if a.block_m <= 0 or M % a.block_m:
            raise ValueError("x must hold whole tiles of block_m rows")
        _need(align_out["tile_expert"], "tile_expert", torch.int32, dev, M // a.block_m)
        a.tile_expert = align_out["tile_expert"].data_ptr()
        layout = (align_out["tile_expert"],)
        if "pair_rows" in align_out:   # ids past the pairs are padding
            _need(align_out["sorted_pair_ids"], "sorted_pair_ids", torch.int32, dev, M)
            a.sorted_pair_ids = align_out["sorted_pair_ids"].data_ptr()
            layout += (align_out["sorted_pair_ids"],)
            held = align_out["pair_rows"].numel()
            a.num_pairs = min(align_out.get("num_pairs", held), held)
    cols = N // 2 if silu_mul else N
    if out is None:
        out = torch.empty((M, cols), dtype=out_dtype or torch.bfloat16, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
        if out.shape != (M, cols):
            raise ValueError(f"out must be {(M, cols)}, got {tuple(out.shape)}")
        _apart(out, x, x_scales, w_codes, w_scales, *layout)
    if M == 0:
        return out
    a.struct_size = ctypes.sizeof(Mx4GemmArgs)
    a.x_dtype = DTYPE_BF16 if x_scales is None else DTYPE_MX4
    a.out_dtype = _row_dtype(out, "out")
    a.num_rows, a.out_features, a.in_features, a.num_experts = M, N, K, E
    a.silu_mul = int(bool(silu_mul))
    a.x, a.w, a.w_scale, a.out = (x.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(),
                                  out.data_ptr())
    a.x_scale = None if x_scales is None else x_scales.data_ptr()
    _launch("moe_lora_mx4_gemm", dev, lib().moe_lora_mx4_gemm, ctypes.byref(a))
    return out


def mx4_block_m(num_tokens: int, top_k: int, num_experts: int) -> int:
    """The block_m of moe_lora_align that suits moe_lora_mx4_gemm: about the rows an
    expert gets, so that its weights are read once without many padding rows.

    Blocks of 64, 128 and 256 rows for 32 experts of 4096 x 7168 with silu_mul, routed at
    random (us): 128 rows an expert 247, 173, 181 of MX4 x and 381, 330, 392 of bf16; 256
    rows 394, 255, 204 and 626, 528, 495; 512 rows 654, 432, 324 and 1128, 945, 841.  256
    is the faster block from about 256 rows an expert on, at up to 255 padding rows an
    expert in every buffer of rows; below 512 rows a caller with the memory for them
    passes it."""
    per = num_tokens * top_k / num_experts
    return 16 if per <= 24 else 32 if per <= 32 else 64 if per <= 128 else 128 if per <= 512 else 256


def run_mx4_layer(inputs: dict, activations: str = "bf16", block_m: Optional[int] = None,
                  out_dtype=None) -> torch.Tensor:
    """The MoE layer without adapters on MX4 expert weights: align -> permute ->
    gate_up product with SiLU * up -> down product -> unpermute.

    ``inputs``: x [T, H] bfloat16, topk_ids, topk_weights, and the weights
    w_gate_up_mx4 [E, 2I, H], w_down_mx4 [E, H, I], each a (codes, scales) pair of
    moe_lora_mx4_quantize.
    ``activations``: "bf16", or "mx4" to quantise x and the activations between the
    products as well.  For serving: there is no gradient, and x or topk_weights that
    require one are refused where autograd is on."""
    if activations not in ("bf16", "mx4"):
        raise ValueError("activations must be 'bf16' or 'mx4'")
    x, ids, w = inputs["x"], inputs["topk_ids"], inputs["topk_weights"]
    if x.requires_grad or (w is not None and w.requires_grad):
        _requires_grad("run_mx4_layer")
    T, k = ids.shape
    gu, down = inputs["w_gate_up_mx4"], inputs["w_down_mx4"]
    H, I = _mx4_pair(*gu, "w_gate_up"), _mx4_pair(*down, "w_down")
    E = gu[0].shape[0]
    if gu[0].shape != (E, 2 * I, H // 2) or down[0].dim() != 3 or down[0].shape[0] != E or x.shape != (T, H):
        raise ValueError(f"x {tuple(x.shape)}, w_gate_up {tuple(gu[0].shape)} and w_down "
                         f"{tuple(down[0].shape)} are not of one layer of {T} tokens: codes "
                         "[E, 2I, H/2] and [E, H, I/2]")
    if block_m is None:
        block_m = mx4_block_m(T, k, E)
    slots = torch.full((max(T, 1),), -1, dtype=torch.int32, device=x.device)
    al = moe_lora_align(ids, slots, None, E, 0, block_m, pair_rows=True)
    if activations == "mx4":
        codes, scales = moe_lora_mx4_quantize(x)
        act = moe_lora_mx4_gemm(moe_lora_permute(codes, al, k), *gu,
                                x_scales=moe_lora_permute(scales, al, k), align_out=al,
                                silu_mul=True)
        codes, scales = moe_lora_mx4_quantize(act, al["num_rows_padded"])
        z = moe_lora_mx4_gemm(codes, *down, x_scales=scales, align_out=al, out_dtype=torch.float32)
    else:
        act = moe_lora_mx4_gemm(moe_lora_permute(x, al, k), *gu, align_out=al, silu_mul=True)
        z = moe_lora_mx4_gemm(act, *down, align_out=al, out_dtype=torch.float32)
    return moe_lora_unpermute(z, al, k, w, out_dtype=out_dtype or x.dtype)
