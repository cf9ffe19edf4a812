"""e4b: NF4 / FP4 quantized Mixture-of-Experts expert kernels for NVIDIA B200.

A thin ctypes binding over ``libe4b.so`` (the C ABI in ``include/e4b.h``).  The
functions keep the C names and only marshal arguments: PyTorch tensors supply
device memory and the current CUDA stream; every step of the computation runs
in the library's sm_100a kernels.  There is no CPU fallback: the first call
fails loudly when the library is missing, and a compute call without a CUDA
device raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# E4B_DEBUG=1 loads the debug-check build (device-side bounds and schedule checks)
DEBUG = os.environ.get("E4B_DEBUG", "0") not in ("", "0")
LIB_PATH = os.path.join(_HERE, "libe4b_debug.so" if DEBUG else "libe4b.so")

E4B_OK, E4B_ERR_INVALID_ARG, E4B_ERR_BLOCKSIZE, E4B_ERR_UNSUPPORTED, E4B_ERR_WORKSPACE, E4B_ERR_CUDA, \
    E4B_ERR_TIMEOUT, E4B_ERR_DEBUG_CHECK = range(8)
# debug-check sites (bits 8..15 of e4b_last_status_word)
SITE_GEMM_TILE, SITE_GEMM_PERM, SITE_GATHER_PERM, SITE_COMBINE_INV, SITE_ROUTER_INV, SITE_OFFSETS, SITE_COUNTS, \
    SITE_TILE_PREFIX, SITE_SCHEDULE, SITE_PERM, SITE_INV_PERM = range(1, 12)
NF4, FP4, MXFP4, INT8, FP8, BF16_WEIGHTS = 0, 1, 2, 3, 4, 5   # storage formats (e4b_codebook)
F32, BF16 = 0, 1
PATH_AUTO, PATH_GROUPED, PATH_DECODE = 0, 1, 2
ACT_SWIGLU, ACT_CLAMPED_GLU = 0, 1
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_ELEMENT = 0, 1, 2, 3                                # e4b_gate
LINEAR_ACT_NONE, LINEAR_ACT_RELU, LINEAR_ACT_SILU, LINEAR_ACT_GELU_TANH = 0, 1, 2, 3   # e4b_linear_act

EXPORTS = ("e4b_quantize_nf4", "e4b_dequantize_nf4", "e4b_quantize_mxfp4", "e4b_dequantize_mxfp4",
           "e4b_mxfp4_scale_stride", "e4b_moe_workspace_size", "e4b_moe_forward",
           "e4b_moe_backward", "e4b_moe_backward_dgrad", "e4b_moe_backward_router", "e4b_device_status", "e4b_status_string",
           "e4b_launch_count", "e4b_timing_enable", "e4b_timing_enable_kinds", "e4b_timing_reset", "e4b_timing_get",
           "e4b_moe_forward_noalloc", "e4b_watchdog_selftest", "e4b_ring_selftest", "e4b_pipe_arena_size", "e4b_pipe_create",
           "e4b_pipe_submit", "e4b_pipe_join", "e4b_pipe_sync", "e4b_pipe_destroy", "e4b_last_status_word",
           "e4b_debug_checks", "e4b_debug_validate_schedule",
           "e4b_moe_dispatch_workspace_size", "e4b_moe_dispatch", "e4b_moe_dispatch_backward", "e4b_moe_combine",
           "e4b_moe_combine_backward", "e4b_block_norm_forward", "e4b_block_norm_workspace_size",
           "e4b_block_norm_backward", "e4b_linear_workspace_size", "e4b_linear_forward_workspace_size",
           "e4b_linear_forward", "e4b_linear_backward")
# kernel kinds of e4b_timing_get
KERNEL_KINDS = ("quantize", "dequantize", "route", "group", "gather", "combine", "gemm_gateup", "gemm_down",
                "gemm_dgrad_down", "gemm_dgrad_gateup", "decode_gateup", "decode_down")


class e4b_moe_desc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int), ("top_k", ctypes.c_int),
                ("renormalize", ctypes.c_int), ("codebook", ctypes.c_int), ("blocksize", ctypes.c_int),
                ("path", ctypes.c_int), ("activation", ctypes.c_int), ("glu_alpha", ctypes.c_float),
                ("glu_limit", ctypes.c_float), ("lora_rank", ctypes.c_int), ("lora_scale", ctypes.c_float)]


class e4b_experts(ctypes.Structure):
    _fields_ = [("gate_up", ctypes.c_void_p), ("down", ctypes.c_void_p), ("gate_up_absmax", ctypes.c_void_p),
                ("down_absmax", ctypes.c_void_p), ("gate_up_bias", ctypes.c_void_p), ("down_bias", ctypes.c_void_p),
                ("lora_A_gu", ctypes.c_void_p), ("lora_B_gu", ctypes.c_void_p), ("lora_A_d", ctypes.c_void_p),
                ("lora_B_d", ctypes.c_void_p), ("gate_up_scales", ctypes.c_void_p), ("down_scales", ctypes.c_void_p)]


class e4b_lora_grads(ctypes.Structure):
    _fields_ = [("dA_gu", ctypes.c_void_p), ("dB_gu", ctypes.c_void_p), ("dA_d", ctypes.c_void_p),
                ("dB_d", ctypes.c_void_p)]


class e4b_block_desc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("gate", ctypes.c_int), ("gate_sigmoid", ctypes.c_int),
                ("residual_scale", ctypes.c_float)]


class e4b_block_branch(ctypes.Structure):
    _fields_ = [("f", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("inv_perm", ctypes.c_void_p),
                ("topk_w", ctypes.c_void_p), ("top_k", ctypes.c_int)]


class e4b_linear_desc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("n_in", ctypes.c_int), ("n_out", ctypes.c_int), ("codebook", ctypes.c_int),
                ("blocksize", ctypes.c_int), ("activation", ctypes.c_int)]


class e4b_linear_weights(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("absmax", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class E4BError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{os.path.basename(LIB_PATH)} not built at {LIB_PATH}; run "
                          f"python -m bit_quantized_mixture_nf4_b200.build --all")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.e4b_quantize_nf4.argtypes = [P, i64, i64, i64, i32, i32, P, P, P]
    lib.e4b_dequantize_nf4.argtypes = [P, P, i64, i64, i64, i32, i32, i32, P, P]
    lib.e4b_quantize_mxfp4.argtypes = [P, i64, i64, i64, P, P, P]
    lib.e4b_dequantize_mxfp4.argtypes = [P, P, i64, i64, i64, i32, P, P]
    lib.e4b_mxfp4_scale_stride.argtypes = [i64]
    lib.e4b_mxfp4_scale_stride.restype = i64
    lib.e4b_moe_workspace_size.argtypes = [ctypes.POINTER(e4b_moe_desc), i64]
    lib.e4b_moe_workspace_size.restype = sz
    lib.e4b_moe_forward.argtypes = [ctypes.POINTER(e4b_moe_desc), ctypes.POINTER(e4b_experts), P, i64, P, P, P, P,
                                    P, P, P, P, P, sz, P]
    lib.e4b_moe_backward.argtypes = [ctypes.POINTER(e4b_moe_desc), ctypes.POINTER(e4b_experts), P, i64, P, P, P, P,
                                     P, P, P, P, P, P, P, sz, P]
    lib.e4b_moe_backward_dgrad.argtypes = [ctypes.POINTER(e4b_moe_desc), ctypes.POINTER(e4b_experts), P, i64, P, P,
                                           P, P, P, P, sz, P]
    lib.e4b_moe_forward_noalloc.argtypes = [ctypes.POINTER(e4b_moe_desc), ctypes.POINTER(e4b_experts), P, i64, P, P,
                                            P, P, P]
    lib.e4b_moe_backward_router.argtypes = [ctypes.POINTER(e4b_moe_desc), ctypes.POINTER(e4b_experts), P, i64, P, P,
                                            P, P, P, P, P, sz, P]
    lib.e4b_device_status.argtypes = [P]
    lib.e4b_last_status_word.argtypes = []
    lib.e4b_last_status_word.restype = ctypes.c_uint32
    lib.e4b_debug_checks.argtypes = []
    lib.e4b_debug_checks.restype = ctypes.c_int
    lib.e4b_debug_validate_schedule.argtypes = [P, i64, i32, i32, P, P, P, P, i64, P, P, P]
    lib.e4b_debug_validate_schedule.restype = ctypes.c_int
    lib.e4b_watchdog_selftest.argtypes = [P]
    lib.e4b_ring_selftest.argtypes = [P, i32, i32, P, P]
    lib.e4b_status_string.argtypes = [i32]
    lib.e4b_status_string.restype = ctypes.c_char_p
    lib.e4b_launch_count.restype = ctypes.c_uint64
    lib.e4b_timing_enable.argtypes = [i32]
    lib.e4b_timing_enable.restype = None
    lib.e4b_timing_enable_kinds.argtypes = [ctypes.c_uint32]
    lib.e4b_pipe_arena_size.argtypes = [ctypes.POINTER(e4b_moe_desc), i64]
    lib.e4b_pipe_arena_size.restype = sz
    lib.e4b_pipe_create.argtypes = [ctypes.POINTER(e4b_moe_desc), ctypes.POINTER(e4b_experts), i64, P, sz, P,
                                    ctypes.POINTER(ctypes.c_void_p)]
    lib.e4b_pipe_submit.argtypes = [P, i64, P, P, P, P, P]
    lib.e4b_pipe_join.argtypes = [P]
    lib.e4b_pipe_sync.argtypes = [P]
    lib.e4b_pipe_destroy.argtypes = [P]
    lib.e4b_pipe_destroy.restype = None
    lib.e4b_timing_enable_kinds.restype = None
    lib.e4b_timing_reset.restype = None
    lib.e4b_timing_get.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_uint64)]
    lib.e4b_timing_get.restype = ctypes.c_int
    lib.e4b_moe_dispatch_workspace_size.argtypes = [i32, i32, i64]
    lib.e4b_moe_dispatch_workspace_size.restype = sz
    lib.e4b_moe_dispatch.argtypes = [i32, i32, P, P, i32, i64, i32, P, P, P, P, P, sz, P]
    lib.e4b_moe_dispatch_backward.argtypes = [P, P, i32, i64, i32, i32, P, P]
    lib.e4b_moe_combine.argtypes = [P, P, P, i32, i64, i32, i32, P, P]
    lib.e4b_moe_combine_backward.argtypes = [P, P, P, P, i32, i64, i32, i32, P, P, P]
    lib.e4b_block_norm_forward.argtypes = [ctypes.POINTER(e4b_block_desc), ctypes.POINTER(e4b_block_branch), P, i64,
                                           P, P, P, P, P, P, P]
    lib.e4b_block_norm_workspace_size.argtypes = [ctypes.POINTER(e4b_block_desc), i64]
    lib.e4b_block_norm_workspace_size.restype = sz
    lib.e4b_block_norm_backward.argtypes = [ctypes.POINTER(e4b_block_desc), P, P, i64] + [P] * 11 + [sz, P]
    lib.e4b_linear_workspace_size.argtypes = [ctypes.POINTER(e4b_linear_desc), i64]
    lib.e4b_linear_workspace_size.restype = sz
    lib.e4b_linear_forward_workspace_size.argtypes = [ctypes.POINTER(e4b_linear_desc), i64]
    lib.e4b_linear_forward_workspace_size.restype = sz
    lib.e4b_linear_forward.argtypes = [ctypes.POINTER(e4b_linear_desc), ctypes.POINTER(e4b_linear_weights), P, i64, P,
                                       P, P, P, P, sz, P]
    lib.e4b_linear_backward.argtypes = [ctypes.POINTER(e4b_linear_desc), ctypes.POINTER(e4b_linear_weights), P, i64, P,
                                        P, P, P, P, P, sz, P]
    for f in ("e4b_quantize_nf4", "e4b_dequantize_nf4", "e4b_quantize_mxfp4", "e4b_dequantize_mxfp4",
              "e4b_moe_forward", "e4b_moe_backward", "e4b_moe_backward_dgrad",
              "e4b_device_status", "e4b_moe_forward_noalloc", "e4b_moe_backward_router", "e4b_watchdog_selftest",
              "e4b_ring_selftest"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def __getattr__(name):
    if name == "lib":
        return _load()
    raise AttributeError(name)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn: str, status: int):
    if status != E4B_OK:
        raise E4BError(fn, status, _load().e4b_status_string(status).decode())


def _new(shape, dtype, device, stream):
    """A tensor for a call on `stream` (None: the current one).  It comes from that stream's memory: a
    block of the current stream's could still be in use by work queued there, which `stream` does not
    wait for.  The current stream may use the tensor too (after waiting for `stream`): its memory is not
    handed out again before what is queued there when it is dropped."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if t.numel():
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _cuda(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def e4b_status_string(status: int) -> str:
    return _load().e4b_status_string(status).decode()


def e4b_launch_count() -> int:
    return int(_load().e4b_launch_count())


def e4b_timing_enable(on: bool = True):
    _load().e4b_timing_enable(int(bool(on)))


def e4b_timing_enable_kinds(kinds):
    """Time only the given kernel kinds (indices or names in KERNEL_KINDS); empty turns timing off."""
    mask = 0
    for k in kinds:
        mask |= 1 << (KERNEL_KINDS.index(k) if isinstance(k, str) else int(k))
    _load().e4b_timing_enable_kinds(mask)


def e4b_timing_reset():
    _load().e4b_timing_reset()


def e4b_timing_get(kind) -> tuple:
    """(total device ms, timed launches) of one kernel kind (index or name in KERNEL_KINDS)."""
    if isinstance(kind, str):
        kind = KERNEL_KINDS.index(kind)
    ms, n = ctypes.c_double(), ctypes.c_uint64()
    _check("e4b_timing_get", _load().e4b_timing_get(kind, ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, int(n.value)


def e4b_device_status(stream=None) -> int:
    return int(_load().e4b_device_status(_stream(stream)))


def e4b_last_status_word() -> int:
    """Raw status word of the last e4b_device_status call (bits 8..15: debug-check site)."""
    return int(_load().e4b_last_status_word())


def e4b_debug_checks() -> bool:
    """True when the loaded library is the debug-check build."""
    return bool(_load().e4b_debug_checks())


def e4b_debug_validate_schedule(topk_idx, E: int, tile_rows: int, counts, offsets, tile_prefix, sched, perm, inv_perm,
                                stream=None) -> int:
    """Checks a grouping schedule on the device; returns the status (E4B_OK or
    E4B_ERR_DEBUG_CHECK, the failing site then in e4b_last_status_word() >> 8)."""
    for t, n in ((topk_idx, "topk_idx"), (counts, "counts"), (offsets, "offsets"), (tile_prefix, "tile_prefix"),
                 (sched, "sched"), (perm, "perm"), (inv_perm, "inv_perm")):
        _cuda(t, n, torch.int32)
    if sched.dim() != 2 or sched.shape[1] != 4:
        raise ValueError("sched must be [n, 4] int32")
    return int(_load().e4b_debug_validate_schedule(_ptr(topk_idx), topk_idx.numel(), E, tile_rows, _ptr(counts),
                                                   _ptr(offsets), _ptr(tile_prefix), _ptr(sched), sched.shape[0],
                                                   _ptr(perm), _ptr(inv_perm), _stream(stream)))


def e4b_quantize_nf4(w: torch.Tensor, blocksize: int = 64, codebook: int = NF4, packed=None, absmax=None,
                     stream=None):
    """w: fp32 [E, out, in] on the GPU -> (packed uint8 [E, out*in/2] (the 8-bit
    codebooks INT8 / FP8: [E, out*in], one byte per element), absmax fp32 [E, out*in/64])."""
    _cuda(w, "w", torch.float32)
    if w.dim() != 3:
        raise ValueError("w must be a 3-D [E, out, in] stack")
    E, o, i = w.shape
    if packed is None:
        packed = _new((E, o * i // (1 if codebook in (INT8, FP8) else 2)), torch.uint8, w.device, stream)
    if absmax is None:
        absmax = _new((E, o * i // max(blocksize, 1)), torch.float32, w.device, stream)
    _check("e4b_quantize_nf4", _load().e4b_quantize_nf4(_ptr(w), E, o, i, blocksize, codebook, _ptr(packed), _ptr(absmax),
                                                    _stream(stream)))
    return packed, absmax


def e4b_dequantize_nf4(packed: torch.Tensor, absmax: torch.Tensor, shape, blocksize: int = 64, codebook: int = NF4,
                       out_dtype: int = BF16, out=None, stream=None):
    """Packed + absmax -> [E, out, in] bf16 (out_dtype=BF16) or fp32 (F32)."""
    _cuda(packed, "packed", torch.uint8)
    _cuda(absmax, "absmax", torch.float32)
    E, o, i = shape
    if out is None:
        out = _new((E, o, i), torch.bfloat16 if out_dtype == BF16 else torch.float32, packed.device, stream)
    _check("e4b_dequantize_nf4", _load().e4b_dequantize_nf4(_ptr(packed), _ptr(absmax), E, o, i, blocksize, codebook,
                                                        out_dtype, _ptr(out), _stream(stream)))
    return out


def make_desc(E, H, I, top_k, renormalize=True, codebook=NF4, blocksize=64, path=PATH_AUTO, activation=ACT_SWIGLU,
              glu_alpha=1.702, glu_limit=7.0, lora_rank=0, lora_scale=1.0) -> e4b_moe_desc:
    return e4b_moe_desc(E, H, I, top_k, int(bool(renormalize)), codebook, blocksize, path, activation, glu_alpha,
                        glu_limit, lora_rank, lora_scale)


def e4b_mxfp4_scale_stride(cols: int) -> int:
    return int(_load().e4b_mxfp4_scale_stride(cols))


def e4b_quantize_mxfp4(w: torch.Tensor, stream=None):
    """fp32 [E, out, in] (CUDA) -> (packed uint8 [E, out*in/2], scales uint8 [E, out, S]):
    OCP MX v1.0 MXFP4 (32-element blocks, E8M0 scales, E2M1 codes)."""
    _cuda(w, "w", torch.float32)
    if w.dim() != 3 or not w.is_contiguous():
        raise ValueError("w must be a contiguous [E, out, in] tensor")
    E, o, i = w.shape
    packed = _new((E, o * i // 2), torch.uint8, w.device, stream)
    scales = _new((E, o, e4b_mxfp4_scale_stride(i)), torch.uint8, w.device, stream)
    _check("e4b_quantize_mxfp4", _load().e4b_quantize_mxfp4(_ptr(w), E, o, i, _ptr(packed), _ptr(scales),
                                                          _stream(stream)))
    return packed, scales


def e4b_dequantize_mxfp4(packed: torch.Tensor, scales: torch.Tensor, shape, out_dtype=torch.bfloat16, stream=None):
    _cuda(packed, "packed", torch.uint8)
    _cuda(scales, "scales", torch.uint8)
    E, o, i = shape
    out = _new((E, o, i), out_dtype, packed.device, stream)
    _check("e4b_dequantize_mxfp4", _load().e4b_dequantize_mxfp4(
        _ptr(packed), _ptr(scales), E, o, i, BF16 if out_dtype == torch.bfloat16 else F32, _ptr(out),
        _stream(stream)))
    return out


def make_experts(gate_up, down, gate_up_absmax, down_absmax, gate_up_bias=None, down_bias=None,
                 lora=None, gate_up_scales=None, down_scales=None) -> e4b_experts:
    """The two packed stacks and their absmax (device tensors), plus optional fp32
    per-expert biases gate_up_bias [E, 2I] and down_bias [E, H], and optional bf16
    LoRA adapters lora = (A_gu [E, r, H], B_gu [E, 2I, r], A_d [E, r, I], B_d [E, H, r])
    (the descriptor's lora_rank must be r).  The tensors must outlive every call
    that uses the returned struct."""
    for n, t in (("gate_up", gate_up), ("down", down)):
        _cuda(t, n, torch.uint8)
    for n, t in (("gate_up_absmax", gate_up_absmax), ("down_absmax", down_absmax)):
        if t is not None:
            _cuda(t, n, torch.float32)
    for n, t in (("gate_up_scales", gate_up_scales), ("down_scales", down_scales)):
        if t is not None:
            _cuda(t, n, torch.uint8)
    for n, t in (("gate_up_bias", gate_up_bias), ("down_bias", down_bias)):
        if t is not None:
            _cuda(t, n, torch.float32)
    ad = [None] * 4
    if lora is not None:
        for i, (n, t) in enumerate(zip(("A_gu", "B_gu", "A_d", "B_d"), lora)):
            _cuda(t, n, torch.bfloat16)
            if not t.is_contiguous():
                raise ValueError(f"{n} must be contiguous")
            ad[i] = t.data_ptr()
    ptr = lambda t: None if t is None else t.data_ptr()
    return e4b_experts(gate_up.data_ptr(), down.data_ptr(), ptr(gate_up_absmax), ptr(down_absmax),
                       ptr(gate_up_bias), ptr(down_bias), *ad, ptr(gate_up_scales), ptr(down_scales))


def e4b_moe_workspace_size(desc: e4b_moe_desc, T: int) -> int:
    return int(_load().e4b_moe_workspace_size(ctypes.byref(desc), T))


def workspace(desc: e4b_moe_desc, T: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(e4b_moe_workspace_size(desc, T), 1), dtype=torch.uint8, device=device)


def e4b_moe_forward(desc: e4b_moe_desc, experts: e4b_experts, x: torch.Tensor, router_logits=None, topk_idx=None,
                    topk_w=None, y=None, saved_gu=None, offsets_out=None, perm_out=None, ws=None, stream=None,
                    saved_h=None):
    """Expert-layer forward.  With router_logits the layer routes and fills
    topk_idx / topk_w (allocated here when not given); without, they are inputs.
    Returns (y, topk_idx, topk_w)."""
    _cuda(x, "x", torch.bfloat16)
    T = x.shape[0]
    dev = x.device
    if topk_idx is None:
        topk_idx = _new((T, desc.top_k), torch.int32, dev, stream)
    if topk_w is None:
        topk_w = _new((T, desc.top_k), torch.float32, dev, stream)
    if router_logits is not None:
        _cuda(router_logits, "router_logits", torch.float32)
    if y is None:
        y = _new((T, desc.H), torch.bfloat16, dev, stream)
    if ws is None:
        ws = _new((max(e4b_moe_workspace_size(desc, T), 1),), torch.uint8, dev, stream)
    _check("e4b_moe_forward", _load().e4b_moe_forward(
        ctypes.byref(desc), ctypes.byref(experts), _ptr(x), T, _ptr(router_logits), _ptr(topk_idx), _ptr(topk_w),
        _ptr(y), _ptr(saved_gu), _ptr(saved_h), _ptr(offsets_out), _ptr(perm_out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return y, topk_idx, topk_w


def e4b_moe_backward(desc: e4b_moe_desc, experts: e4b_experts, x, topk_idx, topk_w, grad_out, saved_gu=None,
                     saved_h=None, router_logits=None, grad_x=None, grad_topk_w=None, grad_logits=None,
                     want_grad_x=True, want_routing=True, lora_grads=None, ws=None, stream=None):
    """The layer backward in one pass: (grad_x bf16 [T, H] or None, grad_topk_w fp32
    [T, k] or None, grad_logits fp32 [T, E] or None).  The routing-weight gradient
    is fused into the input gradient's down^T GEMM; with saved_gu it needs
    saved_h (both from e4b_moe_forward), without them x is used to recompute.
    lora_grads: fp32 tensors (dA_gu, dB_gu, dA_d, dB_d) shaped like the adapters,
    written with the adapter gradients (needs x)."""
    _cuda(grad_out, "grad_out", torch.bfloat16)
    T = grad_out.shape[0]
    dev = grad_out.device
    if grad_x is None and want_grad_x:
        grad_x = _new((T, desc.H), torch.bfloat16, dev, stream)
    if grad_topk_w is None and want_routing:
        grad_topk_w = _new((T, desc.top_k), torch.float32, dev, stream)
    if router_logits is not None:
        _cuda(router_logits, "router_logits", torch.float32)
        if grad_logits is None and want_routing:
            grad_logits = _new((T, desc.E), torch.float32, dev, stream)
    if ws is None:
        ws = _new((max(e4b_moe_workspace_size(desc, T), 1),), torch.uint8, dev, stream)
    lg = None
    if lora_grads is not None:
        for n, t in zip(("dA_gu", "dB_gu", "dA_d", "dB_d"), lora_grads):
            _cuda(t, n, torch.float32)
        lg = e4b_lora_grads(*[t.data_ptr() for t in lora_grads])
    _check("e4b_moe_backward", _load().e4b_moe_backward(
        ctypes.byref(desc), ctypes.byref(experts), _ptr(x), T, _ptr(router_logits), _ptr(topk_idx), _ptr(topk_w),
        _ptr(grad_out), _ptr(saved_gu), _ptr(saved_h), _ptr(grad_x), _ptr(grad_topk_w), _ptr(grad_logits),
        None if lg is None else ctypes.byref(lg), _ptr(ws), ws.numel(), _stream(stream)))
    return grad_x, grad_topk_w, grad_logits


def e4b_moe_backward_dgrad(desc: e4b_moe_desc, experts: e4b_experts, x, topk_idx, topk_w, grad_out, saved_gu=None,
                           grad_x=None, ws=None, stream=None):
    """Input gradient with routing held constant; returns grad_x bf16 [T, H]."""
    _cuda(grad_out, "grad_out", torch.bfloat16)
    T = grad_out.shape[0]
    dev = grad_out.device
    if grad_x is None:
        grad_x = _new((T, desc.H), torch.bfloat16, dev, stream)
    if ws is None:
        ws = _new((max(e4b_moe_workspace_size(desc, T), 1),), torch.uint8, dev, stream)
    _check("e4b_moe_backward_dgrad", _load().e4b_moe_backward_dgrad(
        ctypes.byref(desc), ctypes.byref(experts), _ptr(x), T, _ptr(topk_idx), _ptr(topk_w), _ptr(grad_out),
        _ptr(saved_gu), _ptr(grad_x), _ptr(ws), ws.numel(), _stream(stream)))
    return grad_x


def e4b_moe_forward_noalloc(desc: e4b_moe_desc, experts: e4b_experts, x: torch.Tensor, router_logits=None,
                            topk_idx=None, topk_w=None, y=None, stream=None):
    """The forward with the library's own fixed scratch (no workspace argument).
    Output tensors are allocated here only when not given.  Returns (y, topk_idx, topk_w)."""
    _cuda(x, "x", torch.bfloat16)
    T = x.shape[0]
    dev = x.device
    if topk_idx is None:
        topk_idx = _new((T, desc.top_k), torch.int32, dev, stream)
    if topk_w is None:
        topk_w = _new((T, desc.top_k), torch.float32, dev, stream)
    if router_logits is not None:
        _cuda(router_logits, "router_logits", torch.float32)
    if y is None:
        y = _new((T, desc.H), torch.bfloat16, dev, stream)
    _check("e4b_moe_forward_noalloc", _load().e4b_moe_forward_noalloc(
        ctypes.byref(desc), ctypes.byref(experts), _ptr(x), T, _ptr(router_logits), _ptr(topk_idx), _ptr(topk_w),
        _ptr(y), _stream(stream)))
    return y, topk_idx, topk_w


def e4b_moe_backward_router(desc: e4b_moe_desc, experts: e4b_experts, x, topk_idx, topk_w, grad_out,
                            router_logits=None, grad_topk_w=None, grad_logits=None, want_logits=True, ws=None,
                            stream=None):
    """Routing gradient with the indices held: (grad_topk_w fp32 [T, k],
    grad_logits fp32 [T, E] or None).  grad_logits needs router_logits."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(grad_out, "grad_out", torch.bfloat16)
    T = x.shape[0]
    dev = x.device
    if grad_topk_w is None:
        grad_topk_w = _new((T, desc.top_k), torch.float32, dev, stream)
    if router_logits is not None:
        _cuda(router_logits, "router_logits", torch.float32)
        if grad_logits is None and want_logits:
            grad_logits = _new((T, desc.E), torch.float32, dev, stream)
    if ws is None:
        ws = _new((max(e4b_moe_workspace_size(desc, T), 1),), torch.uint8, dev, stream)
    _check("e4b_moe_backward_router", _load().e4b_moe_backward_router(
        ctypes.byref(desc), ctypes.byref(experts), _ptr(x), T, _ptr(router_logits), _ptr(topk_idx), _ptr(topk_w),
        _ptr(grad_out), _ptr(grad_topk_w), _ptr(grad_logits), _ptr(ws), ws.numel(), _stream(stream)))
    return grad_topk_w, grad_logits


def e4b_watchdog_selftest(stream=None):
    """Launch the watchdog self-test kernel (a bounded wait that must time out)."""
    _check("e4b_watchdog_selftest", _load().e4b_watchdog_selftest(_stream(stream)))


def e4b_ring_selftest(src: torch.Tensor, lost: int = -1, stream=None) -> torch.Tensor:
    """Two groups read src (fp32 [rows, 128]) through the block norm's ring; row `lost` never counts as
    landed.  int32 [4]: per group the rows read, and those in flight when it gave up (-1: wrong)."""
    _cuda(src, "src", torch.float32)
    if src.dim() != 2 or src.shape[1] != 128:
        raise ValueError("src must be [rows, 128]")
    out = _new((4,), torch.int32, src.device, stream)
    _check("e4b_ring_selftest", _load().e4b_ring_selftest(_ptr(src), src.shape[0], lost, _ptr(out), _stream(stream)))
    return out


# ------------------------------------------------------------- pipelined host-buffer steps

def _host(t: torch.Tensor, name: str, dtype, shape):
    if t.is_cuda or not t.is_pinned():
        raise ValueError(f"{name} must be a page-locked host tensor (pin_memory())")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


def e4b_pipe_arena_size(desc: e4b_moe_desc, T_max: int) -> int:
    return int(_load().e4b_pipe_arena_size(ctypes.byref(desc), T_max))


class e4b_pipe:
    """Handle of a pipelined host-buffer step runner (e4b_pipe_create): owns the
    device arena tensor and keeps the descriptor and expert tensors alive."""

    def __init__(self, handle, arena, desc, experts, T_max):
        self.handle, self.arena, self.desc, self.experts, self.T_max = handle, arena, desc, experts, T_max


def e4b_pipe_create(desc: e4b_moe_desc, experts: e4b_experts, T_max: int, device="cuda", stream=None) -> e4b_pipe:
    size = e4b_pipe_arena_size(desc, T_max)
    if size == 0:
        raise ValueError("invalid descriptor or T_max")
    arena = _new((size,), torch.uint8, device, stream)
    h = ctypes.c_void_p()
    _check("e4b_pipe_create", _load().e4b_pipe_create(ctypes.byref(desc), ctypes.byref(experts), T_max,
                                                      _ptr(arena), size, _stream(stream), ctypes.byref(h)))
    return e4b_pipe(h, arena, desc, experts, T_max)


def e4b_pipe_submit(pipe: e4b_pipe, x, router_logits, grad_out, y, grad_x):
    """Enqueue one batch: pinned host x [T,H] bf16, router_logits [T,E] fp32,
    grad_out [T,H] bf16 in; pinned host y and grad_x [T,H] bf16 out (valid after
    a later e4b_pipe_join/e4b_pipe_sync)."""
    d = pipe.desc
    T = x.shape[0]
    args = (_host(x, "x", torch.bfloat16, (T, d.H)), _host(router_logits, "router_logits", torch.float32, (T, d.E)),
            _host(grad_out, "grad_out", torch.bfloat16, (T, d.H)), _host(y, "y", torch.bfloat16, (T, d.H)),
            _host(grad_x, "grad_x", torch.bfloat16, (T, d.H)))
    _check("e4b_pipe_submit", _load().e4b_pipe_submit(pipe.handle, T, *args))


def e4b_pipe_join(pipe: e4b_pipe):
    _check("e4b_pipe_join", _load().e4b_pipe_join(pipe.handle))


def e4b_pipe_sync(pipe: e4b_pipe):
    _check("e4b_pipe_sync", _load().e4b_pipe_sync(pipe.handle))


def e4b_pipe_destroy(pipe: e4b_pipe):
    if pipe.handle:
        _load().e4b_pipe_destroy(pipe.handle)
        pipe.handle = None


# ------------------------------------------------- operators around the expert layer

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _arg(t, name, dtype, shape, device):
    """Pointer of a contiguous CUDA tensor of this type, shape and device (index); None stays None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _device_of(t, name):
    if t is None or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    return t.get_device()


def _call(name, device, stream, *args):
    """Calls the library's function on `device`, the call's stream as its last argument."""
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(name, device, stream, *args)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device)   # torch.cuda.current_stream() costs 3 us
    elif stream.device.index != device:
        raise ValueError(f"stream must be on cuda:{device}, got {stream.device}")
    else:
        raw = stream.cuda_stream
    status = getattr(_lib or _load(), name)(*args, raw)
    if status:
        _check(name, status)


def _ws_arg(ws, need, device, stream):
    """(pointer, bytes) of the caller's workspace or of a new one, and the tensor to keep until the launch."""
    if ws is None:
        ws = _new((max(need, 1),), torch.uint8, device, stream)
    elif ws.dtype is not torch.uint8 or ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{device}")
    return ws.data_ptr(), ws.numel(), ws


def e4b_moe_dispatch_workspace_size(E: int, top_k: int, T: int) -> int:
    return int(_load().e4b_moe_dispatch_workspace_size(E, top_k, T))


def dispatch_workspace(E: int, top_k: int, T: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(e4b_moe_dispatch_workspace_size(E, top_k, T), 1), dtype=torch.uint8, device=device)


def e4b_moe_dispatch(E: int, topk_idx: torch.Tensor, x=None, rows=None, offsets=None, perm=None, inv_perm=None,
                     ws=None, stream=None):
    """Tokens sorted by expert: (rows [T*k, H] or None without x, offsets int32 [E+1], perm int32
    [T*k], inv_perm int32 [T, k]).  rows and perm behind offsets[E] are not written."""
    dev = _device_of(topk_idx, "topk_idx")
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, k]")
    T, k = topk_idx.shape
    H, dt = 1, BF16
    if x is not None:
        if x.dim() != 2 or x.dtype not in _DTYPES:
            raise ValueError("x must be a [T, H] tensor of bfloat16 or float32")
        H, dt = x.shape[1], _DTYPES[x.dtype]
        if rows is None:
            rows = _new((T * k, H), x.dtype, dev, stream)
    elif rows is not None:
        raise ValueError("rows needs x")
    if offsets is None:
        offsets = _new((E + 1,), torch.int32, dev, stream)
    if perm is None:
        perm = _new((T * k,), torch.int32, dev, stream)
    if inv_perm is None:
        inv_perm = _new((T, k), torch.int32, dev, stream)
    args = (_arg(topk_idx, "topk_idx", torch.int32, (T, k), dev),
            None if x is None else _arg(x, "x", x.dtype, (T, H), dev), dt, T, H,
            None if x is None else _arg(rows, "rows", x.dtype, (T * k, H), dev),
            _arg(offsets, "offsets", torch.int32, (E + 1,), dev), _arg(perm, "perm", torch.int32, (T * k,), dev),
            _arg(inv_perm, "inv_perm", torch.int32, (T, k), dev))
    wp, wn, keep = _ws_arg(ws, 0 if ws is not None else e4b_moe_dispatch_workspace_size(E, k, T), dev, stream)
    _call("e4b_moe_dispatch", dev, stream, E, k, *args, wp, wn)
    return rows, offsets, perm, inv_perm


def _rows_args(rows, inv_perm, name):
    dev = _device_of(rows, name)
    if rows.dim() != 2 or rows.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a [T*k, H] tensor of bfloat16 or float32")
    if inv_perm.dim() != 2:
        raise ValueError("inv_perm must be [T, k]")
    T, k = inv_perm.shape
    return dev, T, k, rows.shape[1]


def e4b_moe_dispatch_backward(grad_rows: torch.Tensor, inv_perm: torch.Tensor, grad_x=None, stream=None):
    """grad_x[t] = sum_j grad_rows[inv_perm[t, j]]."""
    dev, T, k, H = _rows_args(grad_rows, inv_perm, "grad_rows")
    dt = grad_rows.dtype
    if grad_x is None:
        grad_x = _new((T, H), dt, dev, stream)
    _call("e4b_moe_dispatch_backward", dev, stream, _arg(grad_rows, "grad_rows", dt, (T * k, H), dev),
          _arg(inv_perm, "inv_perm", torch.int32, (T, k), dev), _DTYPES[dt], T, H, k,
          _arg(grad_x, "grad_x", dt, (T, H), dev))
    return grad_x


def e4b_moe_combine(rows: torch.Tensor, inv_perm: torch.Tensor, topk_w=None, y=None, stream=None):
    """y[t] = sum_j topk_w[t, j] * rows[inv_perm[t, j]] (weights 1 without topk_w)."""
    dev, T, k, H = _rows_args(rows, inv_perm, "rows")
    dt = rows.dtype
    if y is None:
        y = _new((T, H), dt, dev, stream)
    _call("e4b_moe_combine", dev, stream, _arg(rows, "rows", dt, (T * k, H), dev),
          _arg(inv_perm, "inv_perm", torch.int32, (T, k), dev), _arg(topk_w, "topk_w", torch.float32, (T, k), dev),
          _DTYPES[dt], T, H, k, _arg(y, "y", dt, (T, H), dev))
    return y


def e4b_moe_combine_backward(rows, inv_perm: torch.Tensor, topk_w, grad_y: torch.Tensor, grad_rows=None,
                             grad_topk_w=None, want_grad_rows=True, want_grad_w=True, stream=None):
    """(grad_rows [T*k, H] or None, grad_topk_w fp32 [T, k] or None); rows is needed for the second only."""
    dev, dt = _device_of(grad_y, "grad_y"), grad_y.dtype
    if dt not in _DTYPES or inv_perm.dim() != 2 or grad_y.dim() != 2:
        raise ValueError("grad_y must be a [T, H] tensor of bfloat16 or float32 and inv_perm [T, k]")
    (T, k), H = inv_perm.shape, grad_y.shape[1]
    if grad_rows is None and want_grad_rows:
        grad_rows = _new((T * k, H), dt, dev, stream)
    if grad_topk_w is None and want_grad_w:
        grad_topk_w = _new((T, k), torch.float32, dev, stream)
    _call("e4b_moe_combine_backward", dev, stream, _arg(rows, "rows", dt, (T * k, H), dev),
          _arg(inv_perm, "inv_perm", torch.int32, (T, k), dev), _arg(topk_w, "topk_w", torch.float32, (T, k), dev),
          _arg(grad_y, "grad_y", dt, (T, H), dev), _DTYPES[dt], T, H, k,
          _arg(grad_rows, "grad_rows", dt, (T * k, H), dev),
          _arg(grad_topk_w, "grad_topk_w", torch.float32, (T, k), dev))
    return grad_rows, grad_topk_w


def make_block_desc(H, dtype=torch.bfloat16, eps=1e-6, weight_offset=0.0, gate=GATE_NONE, gate_sigmoid=False,
                    residual_scale=1.0) -> e4b_block_desc:
    if dtype not in _DTYPES:
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    return e4b_block_desc(H, _DTYPES[dtype], eps, weight_offset, gate, int(bool(gate_sigmoid)), residual_scale)


def _block_gate(desc, T, dt):
    """(dtype, shape) of the descriptor's gate."""
    if desc.gate == GATE_ELEMENT:
        return dt, (T, desc.H)
    return torch.float32, (desc.H,) if desc.gate == GATE_CHANNEL else (T,)


def e4b_block_norm_forward(desc: e4b_block_desc, h: torch.Tensor, f=None, rows=None, inv_perm=None, topk_w=None,
                           post_w=None, gate=None, pre_w=None, f_out=None, o=None, n=None, stream=None):
    """Post-norm, gate, scaled residual and the next pre-norm: (o or None without a branch, n or
    None without pre_w).  The branch is f [T, H] or the combine of rows, inv_perm and topk_w."""
    if rows is None and (inv_perm is not None or topk_w is not None):
        raise ValueError("inv_perm and topk_w need rows")
    dev, dt, H = _device_of(h, "h"), torch.bfloat16 if desc.dtype == BF16 else torch.float32, desc.H
    if h.dim() != 2:
        raise ValueError("h must be [T, H]")
    T = h.shape[0]
    if rows is not None:
        if f is not None:
            raise ValueError("the branch is either f or rows")
        if inv_perm is None or inv_perm.dim() != 2:
            raise ValueError("rows needs inv_perm [T, k]")
        k = inv_perm.shape[1]
        branch = e4b_block_branch(None, _arg(rows, "rows", dt, (T * k, H), dev),
                                  _arg(inv_perm, "inv_perm", torch.int32, (T, k), dev),
                                  _arg(topk_w, "topk_w", torch.float32, (T, k), dev), k)
    else:
        branch = None if f is None else e4b_block_branch(_arg(f, "f", dt, (T, H), dev))
    if o is None and branch is not None:
        o = _new((T, H), dt, dev, stream)
    if n is None and pre_w is not None:
        n = _new((T, H), dt, dev, stream)
    gd, gs = _block_gate(desc, T, dt)
    _call("e4b_block_norm_forward", dev, stream, desc, branch, _arg(h, "h", dt, (T, H), dev), T,
          _arg(post_w, "post_w", torch.float32, (H,), dev), _arg(gate, "gate", gd, gs, dev),
          _arg(pre_w, "pre_w", torch.float32, (H,), dev), _arg(f_out, "f_out", dt, (T, H), dev),
          _arg(o, "o", dt, (T, H), dev), _arg(n, "n", dt, (T, H), dev))
    return o, n


def e4b_block_norm_workspace_size(desc: e4b_block_desc, T: int) -> int:
    return int(_load().e4b_block_norm_workspace_size(desc, T))


def block_norm_workspace(desc: e4b_block_desc, T: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(e4b_block_norm_workspace_size(desc, T), 1), dtype=torch.uint8, device=device)


def e4b_block_norm_backward(desc: e4b_block_desc, o=None, f=None, post_w=None, gate=None, pre_w=None, grad_o=None,
                            grad_n=None, grad_h=None, grad_f=None, ws=None, stream=None):
    """The gradients as a dict: grad_h; grad_f, grad_post_w, grad_gate, grad_pre_w where the
    operand is given (else None).  o: the stream that pre_w normed; grad_o / grad_n: the gradients
    that reach o and n."""
    lead = grad_n if grad_n is not None else grad_o
    dev, dt, H = _device_of(lead, "grad_o or grad_n"), torch.bfloat16 if desc.dtype == BF16 else torch.float32, desc.H
    if lead.dim() != 2:
        raise ValueError("the gradients must be [T, H]")
    T = lead.shape[0]
    gd, gs = _block_gate(desc, T, dt)
    if grad_h is None:
        grad_h = _new((T, H), dt, dev, stream)
    if grad_f is None and f is not None:
        grad_f = _new((T, H), dt, dev, stream)
    out = {"grad_h": grad_h, "grad_f": grad_f,
           "grad_post_w": None if post_w is None else _new((H,), torch.float32, dev, stream),
           "grad_gate": None if gate is None else _new(gs, gd, dev, stream),
           "grad_pre_w": None if pre_w is None else _new((H,), torch.float32, dev, stream)}
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    wp, wn, keep = _ws_arg(ws, 0 if ws is not None else e4b_block_norm_workspace_size(desc, T), dev, stream)
    _call("e4b_block_norm_backward", dev, stream, desc, _arg(o, "o", dt, (T, H), dev), _arg(f, "f", dt, (T, H), dev), T,
          _arg(post_w, "post_w", torch.float32, (H,), dev), _arg(gate, "gate", gd, gs, dev),
          _arg(pre_w, "pre_w", torch.float32, (H,), dev), _arg(grad_o, "grad_o", dt, (T, H), dev),
          _arg(grad_n, "grad_n", dt, (T, H), dev), _arg(grad_h, "grad_h", dt, (T, H), dev),
          _arg(grad_f, "grad_f", dt, (T, H), dev), ptr(out["grad_post_w"]), ptr(out["grad_gate"]),
          ptr(out["grad_pre_w"]), wp, wn)
    return out


_WEIGHT_BITS = {NF4: 4, FP4: 4, MXFP4: 4, INT8: 8, FP8: 8, BF16_WEIGHTS: 16}


def make_linear_desc(n_in, n_out, E=1, codebook=NF4, activation=LINEAR_ACT_NONE, blocksize=None) -> e4b_linear_desc:
    if blocksize is None:
        blocksize = 32 if codebook == MXFP4 else 64
    return e4b_linear_desc(E, n_in, n_out, codebook, blocksize, activation)


def make_linear_weights(weight: torch.Tensor, scale=None, bias=None) -> e4b_linear_weights:
    """The stored stack [E, n_out, n_in] (uint8 codes, or bfloat16), its block scales (fp32
    absmax, or MXFP4's uint8 scales; None for bf16 storage) and an fp32 bias [E, n_out].  The
    handle keeps the tensors alive."""
    dev = _device_of(weight, "weight")
    if weight.dtype not in (torch.uint8, torch.bfloat16):
        raise ValueError(f"weight must be uint8 or bfloat16, got {weight.dtype}")
    for t, name, kinds in ((weight, "weight", None), (scale, "scale", (torch.float32, torch.uint8)),
                           (bias, "bias", (torch.float32,))):
        if t is None:
            continue
        if t.get_device() != dev or not t.is_contiguous() or (kinds and t.dtype not in kinds):
            raise ValueError(f"{name} must be contiguous, on cuda:{dev} and of a type it can be stored in")
    mx = scale is not None and scale.dtype == torch.uint8
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    w = e4b_linear_weights(ptr(weight), None if mx else ptr(scale), ptr(scale) if mx else None, ptr(bias))
    w._tensors, w._fits = (weight, scale, bias), None
    return w


def _linear_weights(desc, w, device):
    """Checks a handle's tensors against the descriptor (once for each descriptor)."""
    key = (desc.E, desc.n_in, desc.n_out, desc.codebook, device)
    if w._fits == key:
        return
    weight, scale, bias = w._tensors
    n = desc.E * desc.n_in * desc.n_out
    if weight.get_device() != device:
        raise ValueError(f"weight must be on cuda:{device}, got {weight.device}")
    if weight.numel() * weight.element_size() * 8 != n * _WEIGHT_BITS.get(desc.codebook, 0):
        raise ValueError("weight does not have the size of the descriptor's stack")
    if desc.codebook == MXFP4:
        good = scale is not None and scale.dtype == torch.uint8 and \
            scale.numel() == desc.E * desc.n_out * e4b_mxfp4_scale_stride(desc.n_in)
    elif desc.codebook == BF16_WEIGHTS:
        good = True
    else:
        good = scale is not None and scale.dtype == torch.float32 and scale.numel() == n // 64
    if not good:
        raise ValueError("scale does not fit the descriptor's storage format and sizes")
    if bias is not None and bias.numel() != desc.E * desc.n_out:
        raise ValueError("bias must be [E, n_out]")
    w._fits = key


def e4b_linear_workspace_size(desc: e4b_linear_desc, P: int) -> int:
    return int(_load().e4b_linear_workspace_size(desc, P))


def e4b_linear_forward_workspace_size(desc: e4b_linear_desc, P: int) -> int:
    return int(_load().e4b_linear_forward_workspace_size(desc, P))


def linear_workspace(desc: e4b_linear_desc, P: int, device="cuda", backward=True) -> torch.Tensor:
    """For calls of up to P rows; backward=False: of the forward alone."""
    size = e4b_linear_workspace_size if backward else e4b_linear_forward_workspace_size
    return torch.empty(max(size(desc, P), 1), dtype=torch.uint8, device=device)


def e4b_linear_forward(desc: e4b_linear_desc, weights: e4b_linear_weights, x: torch.Tensor, offsets=None,
                       residual=None, y=None, saved_d=None, ws=None, stream=None):
    """y = residual + act(x W_e^T + bias_e), bf16 [P, n_out].  saved_d (bf16 [P, n_out]) receives
    act' for the backward.  Rows outside every expert's range are not written."""
    dev = _device_of(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [P, n_in]")
    P, bf = x.shape[0], torch.bfloat16
    _linear_weights(desc, weights, dev)
    if y is None:
        y = _new((P, desc.n_out), bf, dev, stream)
    wp, wn, keep = _ws_arg(ws, 0 if ws is not None else e4b_linear_forward_workspace_size(desc, P), dev, stream)
    _call("e4b_linear_forward", dev, stream, desc, weights, _arg(x, "x", bf, (P, desc.n_in), dev), P,
          _arg(offsets, "offsets", torch.int32, (desc.E + 1,), dev),
          _arg(residual, "residual", bf, (P, desc.n_out), dev), _arg(y, "y", bf, (P, desc.n_out), dev),
          _arg(saved_d, "saved_d", bf, (P, desc.n_out), dev), wp, wn)
    return y


def e4b_linear_backward(desc: e4b_linear_desc, weights: e4b_linear_weights, grad_y: torch.Tensor, x=None, offsets=None,
                        saved_d=None, grad_x=None, grad_bias=None, want_grad_x=True, want_grad_bias=True, ws=None,
                        stream=None):
    """(grad_x bf16 [P, n_in] or None, grad_bias fp32 [E, n_out] or None).  With an activation it needs
    saved_d, or x to recompute it from."""
    dev = _device_of(grad_y, "grad_y")
    if grad_y.dim() != 2:
        raise ValueError("grad_y must be [P, n_out]")
    P, bf = grad_y.shape[0], torch.bfloat16
    _linear_weights(desc, weights, dev)
    if grad_x is None and want_grad_x:
        grad_x = _new((P, desc.n_in), bf, dev, stream)
    if grad_bias is None and want_grad_bias:
        grad_bias = _new((desc.E, desc.n_out), torch.float32, dev, stream)
    wp, wn, keep = _ws_arg(ws, 0 if ws is not None else e4b_linear_workspace_size(desc, P), dev, stream)
    _call("e4b_linear_backward", dev, stream, desc, weights, _arg(x, "x", bf, (P, desc.n_in), dev), P,
          _arg(offsets, "offsets", torch.int32, (desc.E + 1,), dev),
          _arg(grad_y, "grad_y", bf, (P, desc.n_out), dev), _arg(saved_d, "saved_d", bf, (P, desc.n_out), dev),
          _arg(grad_x, "grad_x", bf, (P, desc.n_in), dev),
          _arg(grad_bias, "grad_bias", torch.float32, (desc.E, desc.n_out), dev), wp, wn)
    return grad_x, grad_bias
