"""Thin Python binding of libsegquant.so: the same entry points as
include/segquant.h, taking torch tensors.  Argument marshalling only -- every
step of the computation runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback.  A missing library raises at the first call.

All tensors must be CUDA tensors on the current device; calls are enqueued on
torch's current CUDA stream.  Every call raises SegQuantError unless the
library returned SQ_OK.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import warnings
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

# The library: the release build, or another build of it named by the
# environment variable SQ_LIBRARY (the test suite runs some cases against the
# bounds-checked debug build, libsegquant_debug.so).
LIB_PATH = os.environ.get("SQ_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libsegquant.so")

SQ_OK = 0
SQ_ERR_UNSUPPORTED = -2
SQ_SEG_NONE, SQ_SEG_OUTPUT, SQ_SEG_INPUT = 0, 1, 2
SQ_OUT_BF16, SQ_OUT_F32 = 0, 1
SQ_MAX_SEGMENTS = 64
SQ_FLAG_SINGLE_SCALE = 1
SQ_FLAG_W4 = 2
SQ_FLAG_FP8 = 4

EXPORTED = ("sq_calibrate_act", "sq_quantize_act", "sq_quantize_weight_seg",
            "sq_quantize_weight_w4", "sq_unpack_weight_w4",
            "sq_dualscale_seglinear_gemm", "sq_dualscale_seglinear_gemm_gelu_quant",
            "sq_debug_gemm_s32", "sq_get_device_status",
            "sq_status_string", "sq_version", "sq_debug_timeout_probe",
            "sq_host_pipeline_workspace_bytes", "sq_host_pipeline_create",
            "sq_host_pipeline_destroy", "sq_dualscale_seglinear_host",
            "sq_dualscale_seglinear_host_noalloc", "sq_choose_single_scale",
            "sq_dualscale_seglinear_gemm_ws", "sq_gemm_workspace_bytes", "sq_debug_gemm_s32_ws",
            "sq_debug_bounds_checks", "sq_debug_bounds_probe",
            "sq_quantize_act_plan", "sq_quantize_act_planned",
            "sq_lora_plan_bytes", "sq_lora_plan", "sq_lora_forward", "sq_lora_workspace_bytes",
            "sq_lora_backward",
            "sq_rope_forward", "sq_rope_backward", "sq_rope_frequencies",
            "sq_group_norm_workspace_bytes", "sq_group_norm_forward", "sq_group_norm_backward",
            "sq_input_grad_workspace_bytes", "sq_dualscale_seglinear_input_grad")
SQ_ROPE_INTERLEAVED, SQ_ROPE_HALF = 0, 1
SQ_ROPE_SCALE_NONE, SQ_ROPE_SCALE_LINEAR, SQ_ROPE_SCALE_NTK, SQ_ROPE_SCALE_YARN = 0, 1, 2, 3
SQ_ACT_NONE, SQ_ACT_SILU, SQ_ACT_GELU = 0, 1, 2
SQ_ERR_INVALID_ARG = -1
SQ_ERR_DEVICE_BOUNDS = -9
SQ_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class SegQuantError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class _Segments(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("n_seg", ctypes.c_int32),
                ("offsets", ctypes.POINTER(ctypes.c_int32)), ("n_groups", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


@dataclass
class Segments:
    """SegLinear segment table: mode, boundaries (over N for output mode, over
    K for input mode), the number of activation groups G, and flags
    (SQ_FLAG_SINGLE_SCALE for the single-scale path, SQ_FLAG_W4 for a GEMM whose
    weight operand comes from sq_unpack_weight_w4, SQ_FLAG_FP8 for E4M3 codes in
    the int8 buffers)."""
    mode: int = SQ_SEG_NONE
    offsets: Optional[Sequence[int]] = None
    n_groups: int = 1
    flags: int = 0

    @property
    def P(self) -> int:
        """Activation planes per group: 2 (X^+, X^-), or 1 in single-scale mode."""
        return 1 if self.flags & SQ_FLAG_SINGLE_SCALE else 2

    @property
    def n_seg(self) -> int:
        return 1 if self.offsets is None else len(self.offsets) - 1

    @property
    def S(self) -> int:
        return self.n_seg if self.mode == SQ_SEG_INPUT else 1

    def _c(self):
        offsets = None if self.offsets is None else tuple(map(int, self.offsets))
        return _c_segments(self.mode, offsets, self.n_groups, self.flags)


@functools.lru_cache(maxsize=256)
def _c_segments(mode, offsets, n_groups, flags):
    """The C form of a segment table (the calls only read it) and its array, which
    lives as long as it."""
    if offsets is None:
        arr, n_seg, ptr = None, 1, ctypes.POINTER(ctypes.c_int32)()
    else:
        arr = (ctypes.c_int32 * len(offsets))(*offsets)
        n_seg, ptr = len(offsets) - 1, ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
    return _Segments(mode, n_seg, ptr, n_groups, flags), arr


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsegquant.so (built in-tree by w8a8_gemm_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m w8a8_gemm_b200.build` "
                "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        p, i64 = ctypes.c_void_p, ctypes.c_int64
        seg = ctypes.POINTER(_Segments)
        L.sq_calibrate_act.argtypes = [p, i64, i64, i64, p, seg, p, p]
        L.sq_quantize_act.argtypes = [p, i64, i64, i64, p, p, seg, p, p]
        L.sq_quantize_act_plan.argtypes = [p, i64, p, seg, p, p]
        L.sq_quantize_act_planned.argtypes = [p, i64, i64, i64, p, p, seg, p, p, p]
        L.sq_quantize_weight_seg.argtypes = [p, i64, i64, p, seg, p, p, p]
        L.sq_quantize_weight_w4.argtypes = [p, i64, i64, p, seg, p, p, p]
        L.sq_unpack_weight_w4.argtypes = [p, i64, i64, p, p]
        L.sq_dualscale_seglinear_gemm.argtypes = [p, p, p, p, p, p, ctypes.c_int, i64, i64, i64,
                                                  i64, seg, p]
        L.sq_dualscale_seglinear_gemm_gelu_quant.argtypes = [p, p, p, p, p, i64, i64, i64, seg,
                                                             p, ctypes.c_int32, p, p]
        L.sq_debug_gemm_s32.argtypes = [p, p, i64, i64, i64, seg, p, p]
        L.sq_debug_gemm_s32_ws.argtypes = [p, p, i64, i64, i64, seg, p, p, ctypes.c_size_t, p]
        L.sq_dualscale_seglinear_gemm_ws.argtypes = [p, p, p, p, p, p, ctypes.c_int, i64, i64,
                                                     i64, i64, seg, p, ctypes.c_size_t, p]
        L.sq_gemm_workspace_bytes.argtypes = []
        L.sq_gemm_workspace_bytes.restype = ctypes.c_size_t
        L.sq_get_device_status.argtypes = [p]
        L.sq_choose_single_scale.argtypes = [p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                             ctypes.POINTER(ctypes.c_int32)]
        L.sq_debug_timeout_probe.argtypes = [ctypes.c_uint32, p]
        L.sq_debug_bounds_checks.argtypes = []
        L.sq_debug_bounds_probe.argtypes = [p, i64, p]
        L.sq_host_pipeline_workspace_bytes.argtypes = [i64, i64, i64, ctypes.c_int32,
                                                       ctypes.c_int32]
        L.sq_host_pipeline_workspace_bytes.restype = ctypes.c_size_t
        L.sq_host_pipeline_create.argtypes = [i64, i64, i64, ctypes.c_int32, ctypes.c_int32, p,
                                              ctypes.c_size_t, ctypes.POINTER(p)]
        L.sq_host_pipeline_destroy.argtypes = [p]
        L.sq_dualscale_seglinear_host.argtypes = [p, p, i64, i64, i64, p, p, p, p, p, p,
                                                  ctypes.c_int, i64, i64, seg, p]
        L.sq_dualscale_seglinear_host_noalloc.argtypes = [p, i64, i64, i64, p, p, p, p, p, p,
                                                          ctypes.c_int, i64, i64, seg, p]
        i32, size, dbl = ctypes.c_int32, ctypes.c_size_t, ctypes.c_double
        c_int, f32 = ctypes.c_int, ctypes.c_float
        L.sq_lora_plan_bytes.argtypes = [i64, i32]
        L.sq_lora_plan_bytes.restype = size
        L.sq_lora_plan.argtypes = [p, i64, i32, p, p]
        L.sq_lora_forward.argtypes = [p, i64, p, p, p, p, p, i64, p, i64, c_int, p, p, size, i64,
                                      i64, i64, i32, i32, p]
        L.sq_lora_workspace_bytes.argtypes = [i64, i32, i32, c_int]
        L.sq_lora_workspace_bytes.restype = size
        L.sq_lora_backward.argtypes = [p, i64, p, i64, p, p, p, p, p, p, i64, p, i64, p, p, c_int,
                                       p, size, i64, i64, i64, i32, i32, p]
        for f in (L.sq_rope_forward, L.sq_rope_backward):
            f.argtypes = [p, i64, p, i64, c_int, p, p, p, i32, f32, i64, i32, i32, i32, c_int, p]
        L.sq_rope_frequencies.argtypes = [i32, dbl, c_int, dbl, dbl, dbl, dbl, p, p]
        L.sq_group_norm_workspace_bytes.argtypes = [i64, i64, i64, i64]
        L.sq_group_norm_workspace_bytes.restype = size
        L.sq_group_norm_forward.argtypes = [p, i64, i64, i64, i64, i64, p, p, f32, c_int, p, i64,
                                            p, p, p, size, p]
        L.sq_group_norm_backward.argtypes = [p, i64, p, i64, i64, i64, i64, i64, p, p, p, p,
                                             c_int, p, i64, p, p, c_int, p, size, p]
        L.sq_input_grad_workspace_bytes.argtypes = [i64, i64]
        L.sq_input_grad_workspace_bytes.restype = size
        L.sq_dualscale_seglinear_input_grad.argtypes = [p, i64, p, p, p, seg, p, i64, i64, i64,
                                                        i64, p, size, p]
        L.sq_status_string.argtypes = [ctypes.c_int]
        L.sq_status_string.restype = ctypes.c_char_p
        L.sq_version.argtypes = []
        for f in (L.sq_calibrate_act, L.sq_quantize_act, L.sq_quantize_weight_seg,
                  L.sq_quantize_weight_w4, L.sq_unpack_weight_w4, L.sq_host_pipeline_create,
                  L.sq_host_pipeline_destroy, L.sq_dualscale_seglinear_host,
                  L.sq_dualscale_seglinear_host_noalloc,
                  L.sq_dualscale_seglinear_gemm, L.sq_dualscale_seglinear_gemm_gelu_quant,
                  L.sq_debug_gemm_s32, L.sq_get_device_status, L.sq_choose_single_scale,
                  L.sq_dualscale_seglinear_gemm_ws, L.sq_debug_gemm_s32_ws,
                  L.sq_version, L.sq_debug_timeout_probe, L.sq_debug_bounds_checks,
                  L.sq_debug_bounds_probe, L.sq_quantize_act_plan, L.sq_quantize_act_planned,
                  L.sq_lora_plan, L.sq_lora_forward, L.sq_lora_backward, L.sq_rope_forward,
                  L.sq_rope_backward, L.sq_rope_frequencies, L.sq_group_norm_forward,
                  L.sq_group_norm_backward, L.sq_dualscale_seglinear_input_grad):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


_native = None


def calls_path() -> str:
    from .build import calls_path as path   # here: python -m w8a8_gemm_b200.build imports this
    return path()


def _calls():
    """The compiled calls of the operators around the quantized linear
    (csrc/torch_calls.cpp) on this library, or False (with a warning, once) where
    there are none for this Python and this torch."""
    global _native
    if _native is None:
        L = lib()
        path = calls_path()
        try:
            spec = importlib.util.spec_from_file_location("_sqtorch", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.init(L._handle)
            _native = module
        except (ImportError, OSError, RuntimeError) as e:
            warnings.warn(f"{os.path.basename(path)} cannot be used ({e}): the operators' calls go "
                          "through ctypes; python -m w8a8_gemm_b200.build builds it",
                          RuntimeWarning)
            _native = False
    return _native


def status_string(code: int) -> str:
    return lib().sq_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != SQ_OK:
        raise SegQuantError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t: Optional[torch.Tensor], dtype, name: str, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _rows(x: torch.Tensor):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    return x.shape[0], x.shape[1], x.stride(0)


# --------------------------------------------------------------------- calls
def sq_calibrate_act(x: torch.Tensor, d: Optional[torch.Tensor], seg: Segments,
                     s_act: torch.Tensor) -> torch.Tensor:
    """AMax calibration into s_act fp32 [G][S][2]."""
    _need(x, torch.bfloat16, "x")
    _need(d, torch.float32, "d", optional=True)
    _need(s_act, torch.float32, "s_act")
    M, K, ldx = _rows(x)
    cs, keep = seg._c()
    _check(lib().sq_calibrate_act(_ptr(x), M, K, ldx, _ptr(d), ctypes.byref(cs), _ptr(s_act),
                                  _stream()), "sq_calibrate_act")
    return s_act


def sq_quantize_act(x: torch.Tensor, d: Optional[torch.Tensor], s_act: torch.Tensor,
                    seg: Segments, planes: torch.Tensor,
                    plan: Optional[torch.Tensor] = None) -> torch.Tensor:
    """DualScale quantization of X / d into planes int8 [G][P][M][K]; with a
    plan from sq_quantize_act_plan (same d, s_act, seg), sq_quantize_act_planned."""
    _need(x, torch.bfloat16, "x")
    _need(d, torch.float32, "d", optional=True)
    _need(s_act, torch.float32, "s_act")
    _need(planes, torch.int8, "planes")
    _need(plan, torch.int32, "plan", optional=True)
    M, K, ldx = _rows(x)
    if tuple(planes.shape) != (seg.n_groups, seg.P, M, K) or not planes.is_contiguous():
        raise ValueError(f"planes must be contiguous [{seg.n_groups}, {seg.P}, {M}, {K}]")
    cs, keep = seg._c()
    if plan is None:
        _check(lib().sq_quantize_act(_ptr(x), M, K, ldx, _ptr(d), _ptr(s_act), ctypes.byref(cs),
                                     _ptr(planes), _stream()), "sq_quantize_act")
    else:
        _check(lib().sq_quantize_act_planned(_ptr(x), M, K, ldx, _ptr(d), _ptr(s_act),
                                             ctypes.byref(cs), _ptr(plan), _ptr(planes),
                                             _stream()), "sq_quantize_act_planned")
    return planes


def sq_quantize_act_plan(d: torch.Tensor, s_act: torch.Tensor, seg: Segments,
                         plan: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per (group, channel) bits [G][ceil(K/32)] (int32 storage of the uint32
    words): channels whose codes may skip both quotient corrections."""
    _need(d, torch.float32, "d")
    _need(s_act, torch.float32, "s_act")
    K = d.shape[-1]
    words = (K + 31) // 32
    if plan is None:
        plan = torch.empty(seg.n_groups, words, dtype=torch.int32, device=d.device)
    _need(plan, torch.int32, "plan")
    if tuple(plan.shape) != (seg.n_groups, words) or not plan.is_contiguous():
        raise ValueError(f"plan must be contiguous int32 [{seg.n_groups}, {words}]")
    cs, keep = seg._c()
    _check(lib().sq_quantize_act_plan(_ptr(d), K, _ptr(s_act), ctypes.byref(cs), _ptr(plan),
                                      _stream()), "sq_quantize_act_plan")
    return plan


def sq_quantize_weight_seg(w: torch.Tensor, d: Optional[torch.Tensor], seg: Segments,
                           wq: torch.Tensor, s_w: torch.Tensor):
    """Segment-wise AMax weight quantization: wq int8 [N][K], s_w fp32 [S][N]."""
    _need(w, torch.bfloat16, "w")
    _need(d, torch.float32, "d", optional=True)
    _need(wq, torch.int8, "wq")
    _need(s_w, torch.float32, "s_w")
    if not (w.is_contiguous() and wq.is_contiguous() and s_w.is_contiguous()):
        raise ValueError("w, wq and s_w must be contiguous")
    N, K = w.shape
    cs, keep = seg._c()
    _check(lib().sq_quantize_weight_seg(_ptr(w), N, K, _ptr(d), ctypes.byref(cs), _ptr(wq),
                                        _ptr(s_w), _stream()), "sq_quantize_weight_seg")
    return wq, s_w


def sq_quantize_weight_w4(w: torch.Tensor, d: Optional[torch.Tensor], seg: Segments,
                          wq4: torch.Tensor, s_w: torch.Tensor):
    """W4A8 weight quantization: packed codes wq4 uint8 [N][K/2], s_w fp32 [S][N]."""
    _need(w, torch.bfloat16, "w")
    _need(d, torch.float32, "d", optional=True)
    _need(wq4, torch.uint8, "wq4")
    _need(s_w, torch.float32, "s_w")
    N, K = w.shape
    if not (w.is_contiguous() and wq4.is_contiguous() and s_w.is_contiguous()):
        raise ValueError("w, wq4 and s_w must be contiguous")
    if tuple(wq4.shape) != (N, K // 2):
        raise ValueError(f"wq4 must be [{N}, {K // 2}]")
    cs, keep = seg._c()
    _check(lib().sq_quantize_weight_w4(_ptr(w), N, K, _ptr(d), ctypes.byref(cs), _ptr(wq4),
                                       _ptr(s_w), _stream()), "sq_quantize_weight_w4")
    return wq4, s_w


def sq_unpack_weight_w4(wq4: torch.Tensor, wq: torch.Tensor) -> torch.Tensor:
    """Packed W4 codes -> the int8 GEMM operand wq [N][K] = 16 q."""
    _need(wq4, torch.uint8, "wq4")
    _need(wq, torch.int8, "wq")
    N, K = wq.shape
    if tuple(wq4.shape) != (N, K // 2) or not (wq4.is_contiguous() and wq.is_contiguous()):
        raise ValueError(f"wq4 must be contiguous [{N}, {K // 2}] and wq contiguous [{N}, {K}]")
    _check(lib().sq_unpack_weight_w4(_ptr(wq4), N, K, _ptr(wq), _stream()),
           "sq_unpack_weight_w4")
    return wq


def gemm_workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for sq_dualscale_seglinear_gemm_ws /
    sq_debug_gemm_s32_ws on the current device (reuse it for every call on one
    stream)."""
    nbytes = lib().sq_gemm_workspace_bytes()
    if nbytes == 0:
        raise SegQuantError(-7, "sq_gemm_workspace_bytes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or torch.device("cuda"))


def sq_dualscale_seglinear_gemm(planes: torch.Tensor, wq: torch.Tensor, s_w: torch.Tensor,
                                s_act: torch.Tensor, bias: Optional[torch.Tensor],
                                y: torch.Tensor, seg: Segments,
                                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = sum_i s_w (s+ X^+_i W^_i + s- X^-_i W^_i) + bias into y (bf16 or fp32 [M][N]).
    With `workspace` (gemm_workspace()), the _ws entry point balances the last
    wave of tiles; the result is the same bit for bit."""
    _need(planes, torch.int8, "planes")
    _need(wq, torch.int8, "wq")
    _need(s_w, torch.float32, "s_w")
    _need(s_act, torch.float32, "s_act")
    _need(bias, torch.bfloat16, "bias", optional=True)
    if y.dtype not in (torch.bfloat16, torch.float32) or not y.is_cuda:
        raise ValueError("y must be a CUDA bf16 or fp32 tensor")
    G, P, M, K = planes.shape
    N = wq.shape[0]
    if P != seg.P or wq.shape[1] != K or y.shape[0] != M or y.shape[1] != N or y.stride(1) != 1:
        raise ValueError("shape mismatch between planes [G,P,M,K], wq [N,K] and y [M,N]")
    out = SQ_OUT_BF16 if y.dtype == torch.bfloat16 else SQ_OUT_F32
    cs, keep = seg._c()
    if workspace is None:
        _check(lib().sq_dualscale_seglinear_gemm(_ptr(planes), _ptr(wq), _ptr(s_w), _ptr(s_act),
                                                 _ptr(bias), _ptr(y), out, M, N, K, y.stride(0),
                                                 ctypes.byref(cs), _stream()),
               "sq_dualscale_seglinear_gemm")
    else:
        _need(workspace, torch.uint8, "workspace")
        _check(lib().sq_dualscale_seglinear_gemm_ws(_ptr(planes), _ptr(wq), _ptr(s_w),
                                                    _ptr(s_act), _ptr(bias), _ptr(y), out, M, N,
                                                    K, y.stride(0), ctypes.byref(cs),
                                                    _ptr(workspace), workspace.numel(),
                                                    _stream()),
               "sq_dualscale_seglinear_gemm_ws")
    return y


def sq_dualscale_seglinear_gemm_gelu_quant(planes: torch.Tensor, wq: torch.Tensor,
                                           s_w: torch.Tensor, s_act: torch.Tensor,
                                           bias: Optional[torch.Tensor], seg: Segments,
                                           s_act_next: torch.Tensor, planes_next: torch.Tensor,
                                           single_next: bool = False) -> torch.Tensor:
    """The fused producer: the next layer's planes of bf16(gelu(bf16(y))) into
    planes_next (int8 [1][P'][M][N], P' = 2, or 1 with single_next), with its
    steps s_act_next (fp32 [2] = {s+, s-}).  This layer: one K-segment."""
    _need(planes, torch.int8, "planes")
    _need(wq, torch.int8, "wq")
    _need(s_w, torch.float32, "s_w")
    _need(s_act, torch.float32, "s_act")
    _need(bias, torch.bfloat16, "bias", optional=True)
    _need(s_act_next, torch.float32, "s_act_next")
    _need(planes_next, torch.int8, "planes_next")
    G, P, M, K = planes.shape
    N = wq.shape[0]
    pn = 1 if single_next else 2
    if (P != seg.P or wq.shape[1] != K or s_act_next.numel() != 2
            or tuple(planes_next.shape) != (1, pn, M, N) or not planes_next.is_contiguous()):
        raise ValueError("shape mismatch between planes [G,P,M,K], wq [N,K] and "
                         "planes_next [1,P',M,N]")
    cs, keep = seg._c()
    _check(lib().sq_dualscale_seglinear_gemm_gelu_quant(
        _ptr(planes), _ptr(wq), _ptr(s_w), _ptr(s_act), _ptr(bias), M, N, K, ctypes.byref(cs),
        _ptr(s_act_next), SQ_FLAG_SINGLE_SCALE if single_next else 0, _ptr(planes_next),
        _stream()), "sq_dualscale_seglinear_gemm_gelu_quant")
    return planes_next


def sq_debug_gemm_s32(planes: torch.Tensor, wq: torch.Tensor, seg: Segments,
                      acc: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Raw int32 accumulators [S][P][M][N] of the same tensor-core kernel (with
    `workspace`: the balanced last wave of sq_debug_gemm_s32_ws)."""
    _need(planes, torch.int8, "planes")
    _need(wq, torch.int8, "wq")
    _need(acc, torch.int32, "acc")
    G, P, M, K = planes.shape
    N = wq.shape[0]
    if tuple(acc.shape) != (seg.S, seg.P, M, N) or not acc.is_contiguous():
        raise ValueError(f"acc must be contiguous [{seg.S}, {seg.P}, {M}, {N}]")
    cs, keep = seg._c()
    if workspace is None:
        _check(lib().sq_debug_gemm_s32(_ptr(planes), _ptr(wq), M, N, K, ctypes.byref(cs),
                                       _ptr(acc), _stream()), "sq_debug_gemm_s32")
    else:
        _need(workspace, torch.uint8, "workspace")
        _check(lib().sq_debug_gemm_s32_ws(_ptr(planes), _ptr(wq), M, N, K, ctypes.byref(cs),
                                          _ptr(acc), _ptr(workspace), workspace.numel(),
                                          _stream()), "sq_debug_gemm_s32_ws")
    return acc


class HostPipeline:
    """Streams, events and a device workspace (a torch tensor this object owns)
    for sq_dualscale_seglinear_host: layers with K <= max_K, N <= max_N,
    G <= max_G, P <= max_P, in chunks of chunk_rows rows."""

    def __init__(self, chunk_rows: int, max_K: int, max_N: int, max_G: int = 1, max_P: int = 2,
                 device=None):
        L = lib()
        nbytes = L.sq_host_pipeline_workspace_bytes(chunk_rows, max_K, max_N, max_G, max_P)
        if nbytes == 0:
            raise ValueError("invalid pipeline sizes")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8,
                                     device=device or torch.device("cuda"))
        self._h = ctypes.c_void_p()
        _check(L.sq_host_pipeline_create(chunk_rows, max_K, max_N, max_G, max_P,
                                         _ptr(self.workspace), nbytes, ctypes.byref(self._h)),
               "sq_host_pipeline_create")

    def close(self):
        if self._h:
            _check(lib().sq_host_pipeline_destroy(self._h), "sq_host_pipeline_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sq_dualscale_seglinear_host(pl: HostPipeline, x_host: torch.Tensor, d: Optional[torch.Tensor],
                                s_act: torch.Tensor, wq: torch.Tensor, s_w: torch.Tensor,
                                bias: Optional[torch.Tensor], y_host: torch.Tensor,
                                seg: Segments) -> torch.Tensor:
    """One layer from host rows x_host (bf16 [M][K], CPU, pinned for overlap)
    to host rows y_host (bf16 or fp32 [M][N], CPU) through the pipeline; the
    weights and scales are CUDA tensors.  Ordered on torch's current stream."""
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("x_host and y_host must be CPU tensors")
    if x_host.dtype != torch.bfloat16 or y_host.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x_host must be bf16 and y_host bf16 or fp32")
    _need(d, torch.float32, "d", optional=True)
    _need(s_act, torch.float32, "s_act")
    _need(wq, torch.int8, "wq")
    _need(s_w, torch.float32, "s_w")
    _need(bias, torch.bfloat16, "bias", optional=True)
    M, K, ldx = _rows(x_host)
    N = wq.shape[0]
    if wq.shape[1] != K or y_host.shape[0] != M or y_host.shape[1] != N or y_host.stride(1) != 1:
        raise ValueError("shape mismatch between x_host [M,K], wq [N,K] and y_host [M,N]")
    out = SQ_OUT_BF16 if y_host.dtype == torch.bfloat16 else SQ_OUT_F32
    cs, keep = seg._c()
    _check(lib().sq_dualscale_seglinear_host(pl._h, _ptr(x_host), M, K, ldx, _ptr(d), _ptr(s_act),
                                             _ptr(wq), _ptr(s_w), _ptr(bias), _ptr(y_host), out,
                                             N, y_host.stride(0), ctypes.byref(cs), _stream()),
           "sq_dualscale_seglinear_host")
    return y_host


def sq_dualscale_seglinear_host_noalloc(x_host: torch.Tensor, d: Optional[torch.Tensor],
                                        s_act: torch.Tensor, wq: torch.Tensor,
                                        s_w: torch.Tensor, bias: Optional[torch.Tensor],
                                        y_host: torch.Tensor, seg: Segments) -> torch.Tensor:
    """The layer of sq_dualscale_seglinear_host without a pipeline or a
    workspace: for callers that may not allocate device memory.  The library's
    fixed device scratch (SQ_NOALLOC_SCRATCH_BYTES) holds the chunks; every
    call on a device shares it, so calls must not overlap on the GPU.  Ordered
    on torch's current stream."""
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("x_host and y_host must be CPU tensors")
    if x_host.dtype != torch.bfloat16 or y_host.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x_host must be bf16 and y_host bf16 or fp32")
    _need(d, torch.float32, "d", optional=True)
    _need(s_act, torch.float32, "s_act")
    _need(wq, torch.int8, "wq")
    _need(s_w, torch.float32, "s_w")
    _need(bias, torch.bfloat16, "bias", optional=True)
    M, K, ldx = _rows(x_host)
    N = wq.shape[0]
    if wq.shape[1] != K or y_host.shape[0] != M or y_host.shape[1] != N or y_host.stride(1) != 1:
        raise ValueError("shape mismatch between x_host [M,K], wq [N,K] and y_host [M,N]")
    out = SQ_OUT_BF16 if y_host.dtype == torch.bfloat16 else SQ_OUT_F32
    cs, keep = seg._c()
    _check(lib().sq_dualscale_seglinear_host_noalloc(_ptr(x_host), M, K, ldx, _ptr(d),
                                                     _ptr(s_act), _ptr(wq), _ptr(s_w), _ptr(bias),
                                                     _ptr(y_host), out, N, y_host.stride(0),
                                                     ctypes.byref(cs), _stream()),
           "sq_dualscale_seglinear_host_noalloc")
    return y_host


# ------------------------------------------- operators around the quantized linear
# These calls are short on the GPU (a few microseconds for a decoding step), so
# they go through compiled checks (_calls) where those are built.  What follows
# them in each function is the same call through ctypes: it runs where they are
# not built, and finds the reason where they say that an argument does not fit.
# One comparison per tensor, and an explanation looked for only when it fails.
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_OUT = {_BF16: SQ_OUT_BF16, _F32: SQ_OUT_F32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _done(r, where: str):
    """The outputs of a compiled call, which returns an int where the library
    refused it."""
    if r.__class__ is int:
        _check(r, where)
    return r


def _explain(name: str, t, dtype, shape, dev: int, contiguous: bool):
    """Raises the reason for which t is not a tensor of this type and shape, with
    contiguous elements (or unit column stride), on device `dev`."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required" if t is None else f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have unit column stride")


def _whole(name: str, t, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on device `dev`."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == dev):
            return t.data_ptr()
    except AttributeError:
        pass
    _explain(name, t, dtype, shape, dev, True)


def _matrix(name: str, t, dtype, shape, dev: int):
    """(address, leading dimension) of a tensor of rows with unit column stride; a
    single row's stride says nothing: its length up to a multiple of 8 is taken."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            ld, unit = t.stride()
            if shape[0] <= 1:
                ld = (shape[1] + 7) // 8 * 8
            if unit == 1 or shape[1] <= 1 or shape[0] == 0:
                return t.data_ptr(), ld
    except AttributeError:
        pass
    _explain(name, t, dtype, shape, dev, False)


def _is_tensor(name: str, t, dev: int):
    """Raises unless t is a tensor (of which type and shape is checked later)."""
    if not isinstance(t, torch.Tensor):
        _explain(name, t, None, (), dev, False)


def _rows_of(name: str, t, dtype):
    """(rows, columns, device) of the tensor that gives a call its sizes."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _explain(name, t, dtype, (), -1, False)
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, not on the current device")
    try:
        rows, cols = t.shape
    except ValueError:
        raise ValueError(f"{name} must have two dimensions") from None
    return rows, cols, dev


def _out_dtype(dtype, name: str) -> int:
    """The ABI's number of a type, bf16 or fp32."""
    if dtype not in _OUT:
        raise ValueError(f"{name} must be bf16 or fp32, got {dtype}")
    return _OUT[dtype]


def _stream_on(dev: int) -> int:
    """torch's current stream on a device whose tensors exist (CUDA is up)."""
    return (_raw_stream(dev) if _raw_stream is not None
            else torch.cuda.current_stream(dev).cuda_stream)


def _workspace(t, nbytes: int, dev: int):
    """(tensor, address, bytes) of the caller's workspace or a new one.  A new one
    is freed when the call returns: torch hands its memory out again to later
    work of the same stream only."""
    if t is None:
        t = torch.empty(nbytes, dtype=_U8, device=dev)
    elif (not isinstance(t, torch.Tensor) or t.dtype is not _U8 or not t.is_contiguous()
          or t.get_device() != dev):
        raise ValueError("workspace must be a contiguous uint8 tensor on the call's device")
    return t, t.data_ptr(), t.numel()


@functools.lru_cache(maxsize=512)
def sq_lora_plan_bytes(M: int, n_adapters: int) -> int:
    """Bytes of the plan of M rows and n_adapters adapters (0: out of range)."""
    return lib().sq_lora_plan_bytes(M, n_adapters)


def sq_lora_plan(adapter: torch.Tensor, n_adapters: int,
                 plan: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The plan of a batch whose row m has adapter[m] (int32 [M]; outside
    0 .. n_adapters - 1: none).  One plan serves all adapted layers of the batch."""
    _need(adapter, _I32, "adapter")
    if adapter.dim() != 1:
        raise ValueError("adapter must have one dimension")
    M, dev = adapter.shape[0], adapter.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"adapter is on cuda:{dev}, not on the current device")
    nbytes = sq_lora_plan_bytes(M, n_adapters)
    if nbytes == 0:
        raise SegQuantError(SQ_ERR_INVALID_ARG, "sq_lora_plan")
    if plan is None:
        plan = torch.empty(nbytes // 4, dtype=_I32, device=dev)
    _check(lib().sq_lora_plan(_whole("adapter", adapter, _I32, (M,), dev), M, n_adapters,
                              _whole("plan", plan, _I32, (nbytes // 4,), dev),
                              _stream_on(dev)), "sq_lora_plan")
    return plan


@functools.lru_cache(maxsize=512)
def sq_lora_workspace_bytes(M: int, R: int, n_adapters: int, dtype=torch.bfloat16) -> int:
    """Workspace bytes of sq_lora_forward (dtype of y) and sq_lora_backward (0:
    sizes out of range)."""
    return lib().sq_lora_workspace_bytes(M, R, n_adapters, _out_dtype(dtype, "dtype"))


def _lora_sizes(A, B):
    """(L, R, K, N) of A [L, R, K] and B [L, N, R]."""
    try:
        L, R, K = A.shape
        _, N, _ = B.shape
        return L, R, K, N
    except (AttributeError, ValueError):
        raise ValueError("A must be [L, R, K] and B [L, N, R]") from None


def sq_lora_forward(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                    plan: torch.Tensor, base: Optional[torch.Tensor],
                    y: Optional[torch.Tensor] = None, t: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """y = base + scale[a] B[a] (A[a] x) per row with adapter a -> (y, t).  base
    bf16 or fp32 [M, N] (None: zeros, bf16 unless y says otherwise); y may be base
    (in place); t fp32 [M, R] is kept for the backward pass (rows without an
    adapter are not written)."""
    native = _native or _calls()
    if native:
        r = native.lora_forward(x, A, B, scale, plan, base, y, t, workspace)
        if r is not None:
            return _done(r, "sq_lora_forward")
    M, K, dev = _rows_of("x", x, _BF16)
    L, R, Ka, N = _lora_sizes(A, B)
    if Ka != K:
        raise ValueError(f"A has K = {Ka}, x has {K}")
    for name, given in (("base", base), ("y", y)):
        if given is not None:
            _is_tensor(name, given, dev)
    if y is None:
        y = torch.empty(M, N, dtype=_BF16 if base is None else base.dtype, device=dev)
    if t is None:
        t = torch.empty(M, R, dtype=_F32, device=dev)
    kind = y.dtype
    out = _out_dtype(kind, "y")
    ws, wp, wn = _workspace(workspace, sq_lora_workspace_bytes(M, R, L, kind)
                            if workspace is None else 0, dev)
    px, ldx = _matrix("x", x, _BF16, (M, K), dev)
    pb, ldb = (None, 0) if base is None else _matrix("base", base, kind, (M, N), dev)
    py, ldy = _matrix("y", y, kind, (M, N), dev)
    _check(lib().sq_lora_forward(
        px, ldx, _whole("A", A, _BF16, (L, R, K), dev), _whole("B", B, _BF16, (L, N, R), dev),
        _whole("scale", scale, _F32, (L,), dev),
        _whole("plan", plan, _I32, (sq_lora_plan_bytes(M, L) // 4,), dev), pb, ldb, py, ldy, out,
        _whole("t", t, _F32, (M, R), dev), wp, wn, M, N, K, R, L, _stream_on(dev)),
        "sq_lora_forward")
    return y, t


def sq_lora_backward(dy: torch.Tensor, x: torch.Tensor, t: torch.Tensor, A: torch.Tensor,
                     B: torch.Tensor, scale: torch.Tensor, plan: torch.Tensor,
                     dx_base: Optional[torch.Tensor], dx: Optional[torch.Tensor] = None,
                     dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                     grad_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                     need_dx: bool = True, need_weights: bool = True):
    """Gradients of sq_lora_forward -> (dA, dB, dx): dA [L, R, K] and dB [L, N, R]
    of grad_dtype (bf16 or fp32; None without need_weights), dx = dx_base + the
    adapters' part (dx_base None: zeros; dx may be dx_base; None without need_dx)."""
    native = _native or _calls()
    if native and grad_dtype in _OUT:
        r = native.lora_backward(dy, x, t, A, B, scale, plan, dx_base, dx, dA, dB,
                                 grad_dtype is _F32, workspace, need_dx, need_weights)
        if r is not None:
            return _done(r, "sq_lora_backward")
    M, N, dev = _rows_of("dy", dy, _BF16)
    L, R, K, Nb = _lora_sizes(A, B)
    if Nb != N:
        raise ValueError(f"B has N = {Nb}, dy has {N}")
    out = _out_dtype(grad_dtype, "grad_dtype")
    pb, ldb, pd, ldd, pA, pB = None, 0, None, 0, None, None
    if need_dx:
        if dx is None:
            dx = torch.empty(M, K, dtype=_BF16, device=dev)
        pd, ldd = _matrix("dx", dx, _BF16, (M, K), dev)
        if dx_base is not None:
            pb, ldb = _matrix("dx_base", dx_base, _BF16, (M, K), dev)
    elif dx is not None or dx_base is not None:
        raise ValueError("dx and dx_base are of no use without need_dx")
    if need_weights:
        if dA is None:
            dA = torch.empty(L, R, K, dtype=grad_dtype, device=dev)
        if dB is None:
            dB = torch.empty(L, N, R, dtype=grad_dtype, device=dev)
        pA = _whole("dA", dA, grad_dtype, (L, R, K), dev)
        pB = _whole("dB", dB, grad_dtype, (L, N, R), dev)
    elif dA is not None or dB is not None:
        raise ValueError("dA and dB are of no use without need_weights")
    ws, wp, wn = _workspace(workspace, sq_lora_workspace_bytes(M, R, L, grad_dtype)
                            if workspace is None else 0, dev)
    pdy, lddy = _matrix("dy", dy, _BF16, (M, N), dev)
    px, ldx = _matrix("x", x, _BF16, (M, K), dev)
    _check(lib().sq_lora_backward(
        pdy, lddy, px, ldx, _whole("t", t, _F32, (M, R), dev),
        _whole("A", A, _BF16, (L, R, K), dev), _whole("B", B, _BF16, (L, N, R), dev),
        _whole("scale", scale, _F32, (L,), dev),
        _whole("plan", plan, _I32, (sq_lora_plan_bytes(M, L) // 4,), dev), pb, ldb, pd, ldd, pA,
        pB, out, wp, wn, M, N, K, R, L, _stream_on(dev)), "sq_lora_backward")
    return dA, dB, dx


def sq_rope_frequencies(rot: int, base: float = 10000.0, scaling: int = SQ_ROPE_SCALE_NONE,
                        scale: float = 1.0, original_context: float = 0.0,
                        beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq, factor): fp32 CPU tensor [rot / 2] and the factor for the rotary
    calls; evaluated on the host in fp64."""
    if rot < 2 or rot % 2 or rot > 1024:
        raise SegQuantError(SQ_ERR_INVALID_ARG, "sq_rope_frequencies")
    inv_freq = torch.empty(rot // 2, dtype=_F32)
    factor = ctypes.c_float(1.0)
    _check(lib().sq_rope_frequencies(rot, base, scaling, scale, original_context, beta_fast,
                                     beta_slow, inv_freq.data_ptr(), ctypes.byref(factor)),
           "sq_rope_frequencies")
    return inv_freq, factor.value


@functools.lru_cache(maxsize=64)
def _int_array(values: tuple):
    """A C int array of these values (read only by the calls)."""
    return (ctypes.c_int32 * len(values))(*values)


def _rope(call: str, x, positions, inv_freq, head_dim, out, layout, axis_pairs, factor):
    native = _native or _calls()
    if native:
        r = native.rope(call == "sq_rope_backward", x, positions, inv_freq, head_dim, out, layout,
                        axis_pairs, factor)
        if r is not None:
            return _done(r, call)[0]
    kind = getattr(x, "dtype", None)
    if kind is None:
        raise ValueError("x must be a tensor")
    dtype = _out_dtype(kind, "x")
    M, cols, dev = _rows_of("x", x, kind)
    if head_dim < 1 or cols % head_dim != 0:
        raise ValueError(f"{cols} columns are no whole number of heads of {head_dim}")
    axes = 1 if axis_pairs is None else len(axis_pairs)
    flat = axes == 1 and isinstance(positions, torch.Tensor) and positions.dim() == 1
    _is_tensor("inv_freq", inv_freq, dev)
    pairs = inv_freq.numel()
    if out is None:
        out = torch.empty(M, cols, dtype=kind, device=dev)
    px, ldx = _matrix("x", x, kind, (M, cols), dev)
    po, ldo = _matrix("out", out, kind, (M, cols), dev)
    _check(getattr(lib(), call)(px, ldx, po, ldo, dtype,
                                _whole("positions", positions, _I32, (M,) if flat else (M, axes),
                                       dev),
                                _whole("inv_freq", inv_freq, _F32, (pairs,), dev),
                                None if axis_pairs is None else _int_array(tuple(axis_pairs)),
                                axes, factor, M, cols // head_dim, head_dim, 2 * pairs, layout,
                                _stream_on(dev)), call)
    return out


def sq_rope_forward(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                    head_dim: int, out: Optional[torch.Tensor] = None,
                    layout: int = SQ_ROPE_INTERLEAVED, axis_pairs: Optional[Sequence[int]] = None,
                    factor: float = 1.0) -> torch.Tensor:
    """Rotary positions on rows x (bf16 or fp32 [M, H * head_dim], a column slice
    of a wider buffer allowed): the first 2 * len(inv_freq) columns of each head
    turn by positions (int32 [M] or [M, axes]) times inv_freq.  out may be x (in
    place).  axis_pairs: the pairs that turn with each axis."""
    return _rope("sq_rope_forward", x, positions, inv_freq, head_dim, out, layout, axis_pairs,
                 factor)


def sq_rope_backward(dout: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                     head_dim: int, dx: Optional[torch.Tensor] = None,
                     layout: int = SQ_ROPE_INTERLEAVED,
                     axis_pairs: Optional[Sequence[int]] = None,
                     factor: float = 1.0) -> torch.Tensor:
    """The gradient of sq_rope_forward with respect to x; dx may be dout."""
    return _rope("sq_rope_backward", dout, positions, inv_freq, head_dim, dx, layout, axis_pairs,
                 factor)


@functools.lru_cache(maxsize=512)
def sq_group_norm_workspace_bytes(B: int, S: int, C: int, G: int) -> int:
    """Workspace bytes of the group norm calls (0: sizes out of range, or B = 0)."""
    return lib().sq_group_norm_workspace_bytes(B, S, C, G)


def _samples(name: str, t, shape, dev: int):
    """(address, row stride) of a [B, S, C] bf16 tensor whose samples and rows lie
    at one row stride."""
    B, S, C = shape
    if (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.shape == shape
            and t.get_device() == dev):
        sb, sr, sc = t.stride()
        if B * S <= 1:
            return t.data_ptr(), (C + 7) // 8 * 8
        ld = sr if S > 1 else sb
        if (sc == 1 or C == 1) and (B == 1 or S == 1 or sb == S * ld):
            return t.data_ptr(), ld
        raise ValueError(f"{name} must have unit channel stride and one row stride")
    _explain(name, t, _BF16, shape, dev, False)


def _gn_sizes(x):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        _explain("x", x, _BF16, (), -1, False)
    if x.dim() != 3:
        raise ValueError("x must be [B, S, C]")
    dev = x.get_device()
    if dev != _current_device():
        raise ValueError(f"x is on cuda:{dev}, not on the current device")
    return (*x.shape, dev)


def sq_group_norm_forward(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor],
                          beta: Optional[torch.Tensor], eps: float = 1e-5,
                          act: int = SQ_ACT_NONE, y: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None):
    """y = act(group norm of x) over channels-last samples x bf16 [B, S, C] ->
    (y, mean, rstd); mean and rstd fp32 [B, groups] are kept for the backward
    pass.  gamma, beta bf16 [C] or None; y may be x (in place)."""
    native = _native or _calls()
    if native:
        r = native.group_norm_forward(x, groups, gamma, beta, eps, act, y, workspace)
        if r is not None:
            return _done(r, "sq_group_norm_forward")
    B, S, C, dev = _gn_sizes(x)
    if y is None:
        y = torch.empty(B, S, C, dtype=_BF16, device=dev)
    mean, rstd = torch.empty(2, B, min(max(groups, 0), C), dtype=_F32, device=dev).unbind(0)
    ws, wp, wn = _workspace(workspace, sq_group_norm_workspace_bytes(B, S, C, groups)
                            if workspace is None else 0, dev)
    px, ldx = _samples("x", x, (B, S, C), dev)
    py, ldy = _samples("y", y, (B, S, C), dev)
    _check(lib().sq_group_norm_forward(
        px, ldx, B, S, C, groups, None if gamma is None else _whole("gamma", gamma, _BF16, (C,), dev),
        None if beta is None else _whole("beta", beta, _BF16, (C,), dev), eps, act, py, ldy,
        mean.data_ptr(), rstd.data_ptr(), wp, wn, _stream_on(dev)), "sq_group_norm_forward")
    return y, mean, rstd


def sq_group_norm_backward(dy: torch.Tensor, x: torch.Tensor, groups: int,
                           gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                           mean: torch.Tensor, rstd: torch.Tensor, act: int = SQ_ACT_NONE,
                           dx: Optional[torch.Tensor] = None, grad_dtype=torch.bfloat16,
                           workspace: Optional[torch.Tensor] = None, need_dx: bool = True):
    """Gradients of sq_group_norm_forward -> (dx, dgamma, dbeta); dgamma and dbeta
    [C] of grad_dtype (None where gamma or beta is None); dx may be dy."""
    native = _native or _calls()
    if native and grad_dtype in _OUT:
        r = native.group_norm_backward(dy, x, groups, gamma, beta, mean, rstd, act, dx,
                                       grad_dtype is _F32, workspace, need_dx)
        if r is not None:
            return _done(r, "sq_group_norm_backward")
    B, S, C, dev = _gn_sizes(x)
    shape = (B, S, C)
    out = _out_dtype(grad_dtype, "grad_dtype")
    if need_dx and dx is None:
        dx = torch.empty(shape, dtype=_BF16, device=dev)
    if not need_dx and dx is not None:
        raise ValueError("dx is of no use without need_dx")
    dgamma = None if gamma is None else torch.empty(C, dtype=grad_dtype, device=dev)
    dbeta = None if beta is None else torch.empty(C, dtype=grad_dtype, device=dev)
    ws, wp, wn = _workspace(workspace, sq_group_norm_workspace_bytes(B, S, C, groups)
                            if workspace is None else 0, dev)
    pdy, lddy = _samples("dy", dy, shape, dev)
    px, ldx = _samples("x", x, shape, dev)
    pdx, lddx = (None, 0) if dx is None else _samples("dx", dx, shape, dev)
    _check(lib().sq_group_norm_backward(
        pdy, lddy, px, ldx, B, S, C, groups,
        None if gamma is None else _whole("gamma", gamma, _BF16, (C,), dev),
        None if beta is None else _whole("beta", beta, _BF16, (C,), dev),
        _whole("mean", mean, _F32, (B, groups), dev),
        _whole("rstd", rstd, _F32, (B, groups), dev), act, pdx, lddx,
        None if dgamma is None else dgamma.data_ptr(), None if dbeta is None else dbeta.data_ptr(),
        out, wp, wn, _stream_on(dev)), "sq_group_norm_backward")
    return dx, dgamma, dbeta


@functools.lru_cache(maxsize=512)
def sq_input_grad_workspace_bytes(N: int, K: int) -> int:
    """Workspace bytes of sq_dualscale_seglinear_input_grad (0: out of range)."""
    return lib().sq_input_grad_workspace_bytes(N, K)


def sq_dualscale_seglinear_input_grad(dy: torch.Tensor, wq: torch.Tensor, s_w: torch.Tensor,
                                      d: Optional[torch.Tensor], seg: Segments,
                                      dx: Optional[torch.Tensor] = None,
                                      workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx = dy (s_w W^ / d): the gradient of a frozen quantized layer with respect
    to its input (dy bf16 [M, N] -> dx bf16 [M, K]), straight through the
    activation quantizer.  workspace: uint8, sq_input_grad_workspace_bytes(N, K);
    layers on one stream may share one."""
    native = _native or _calls()
    if native:
        cs, keep = seg._c()
        r = native.input_grad(dy, wq, s_w, d, ctypes.addressof(cs), seg.n_groups, seg.S, dx,
                              workspace)
        if r is not None:
            return _done(r, "sq_dualscale_seglinear_input_grad")[0]
    M, N, dev = _rows_of("dy", dy, _BF16)
    if not isinstance(wq, torch.Tensor) or wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    K = wq.shape[1]
    if dx is None:
        dx = torch.empty(M, K, dtype=_BF16, device=dev)
    ws, wp, wn = _workspace(workspace, sq_input_grad_workspace_bytes(N, K)
                            if workspace is None else 0, dev)
    pdy, lddy = _matrix("dy", dy, _BF16, (M, N), dev)
    pdx, lddx = _matrix("dx", dx, _BF16, (M, K), dev)
    cs, keep = seg._c()
    _check(lib().sq_dualscale_seglinear_input_grad(
        pdy, lddy, _whole("wq", wq, torch.int8, (N, K), dev),
        _whole("s_w", s_w, _F32, (seg.S, N), dev),
        None if d is None else _whole("d", d, _F32, (seg.n_groups, K), dev), ctypes.byref(cs),
        pdx, lddx, M, N, K, wp, wn, _stream_on(dev)), "sq_dualscale_seglinear_input_grad")
    return dx


def sq_get_device_status() -> int:
    """Wait for torch's current stream, then return (and clear) the device
    error word (one per device, shared by all streams and callers)."""
    return lib().sq_get_device_status(_stream())


def sq_choose_single_scale(s_act: torch.Tensor, fp8: bool = False,
                           threshold: float = 2.0) -> bool:
    """The adaptive DualScale policy on a layer's calibrated DualScale steps
    (fp32 [G][S][2], any device; copied to the host): True where every group
    and K-segment has its larger side below threshold times the smaller."""
    s = s_act.detach().to("cpu", torch.float32).contiguous()
    if s.dim() < 1 or s.shape[-1] != 2:
        raise ValueError("s_act must end in a dimension of 2 ({s+, s-})")
    out = ctypes.c_int32(0)
    _check(lib().sq_choose_single_scale(ctypes.c_void_p(s.data_ptr()), s.numel() // 2,
                                        SQ_FLAG_FP8 if fp8 else 0, float(threshold),
                                        ctypes.byref(out)), "sq_choose_single_scale")
    return bool(out.value)


def sq_debug_timeout_probe(limit_us: int) -> None:
    """Test only: a kernel whose bounded barrier wait runs out after limit_us;
    the timeout lands in the device error word (see sq_get_device_status)."""
    _check(lib().sq_debug_timeout_probe(int(limit_us), _stream()), "sq_debug_timeout_probe")


def sq_debug_bounds_checks() -> bool:
    """True if the loaded library is the bounds-checked debug build."""
    return lib().sq_debug_bounds_checks() == 1


def sq_debug_bounds_probe(buf: torch.Tensor, n: int) -> None:
    """Test only (debug build): one checked store to buf[n] while the check is
    told the buffer holds n elements; buf must hold n + 1 int32 (a guard).
    The debug build skips the store and records SQ_ERR_DEVICE_BOUNDS."""
    _need(buf, torch.int32, "buf")
    if buf.numel() < n + 1:
        raise ValueError("buf must hold n + 1 elements")
    _check(lib().sq_debug_bounds_probe(_ptr(buf), int(n), _stream()), "sq_debug_bounds_probe")


def sq_version() -> int:
    return lib().sq_version()
