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
import os
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
        if self.offsets is None:
            arr = None
            ptr = ctypes.POINTER(ctypes.c_int32)()
        else:
            arr = (ctypes.c_int32 * len(self.offsets))(*[int(v) for v in self.offsets])
            ptr = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
        s = _Segments(self.mode, self.n_seg, ptr, self.n_groups, self.flags)
        return s, arr  # keep the array alive for the call


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
_OUT = {torch.bfloat16: SQ_OUT_BF16, torch.float32: SQ_OUT_F32}


def _out_dtype(t, name: str) -> int:
    """The ABI's number of a tensor's (or a dtype's) type, bf16 or fp32."""
    dtype = t.dtype if isinstance(t, torch.Tensor) else t
    if dtype not in _OUT:
        raise ValueError(f"{name} must be bf16 or fp32, got {dtype}")
    return _OUT[dtype]


def _here(dev, **tensors):
    """Every given tensor is a CUDA tensor on `dev`, the current device."""
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {dev}, not on the current device")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")


def _shape(t: Optional[torch.Tensor], dtype, shape, name: str, contiguous: bool = True):
    """t (where given) has this type and shape, and is contiguous or, for rows,
    has unit column stride."""
    if t is None:
        return
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not contiguous and t.numel() and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")


def _ld(t: torch.Tensor) -> int:
    """Leading dimension of rows; a single row's stride says nothing."""
    cols = t.shape[1]
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), (cols + 7) // 8 * 8)


def sq_lora_plan_bytes(M: int, n_adapters: int) -> int:
    """Bytes of the plan of M rows and n_adapters adapters (0: out of range)."""
    return lib().sq_lora_plan_bytes(M, n_adapters)


def sq_lora_plan(adapter: torch.Tensor, n_adapters: int,
                 plan: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The plan of a batch whose row m has adapter[m] (int32 [M]; outside
    0 .. n_adapters - 1: none).  One plan serves all adapted layers of the batch."""
    _need(adapter, torch.int32, "adapter")
    if adapter.dim() != 1 or not adapter.is_contiguous():
        raise ValueError("adapter must be a contiguous 1-D tensor")
    _here(adapter.device, plan=plan)
    M = adapter.shape[0]
    nbytes = sq_lora_plan_bytes(M, n_adapters)
    if nbytes == 0:
        raise SegQuantError(SQ_ERR_INVALID_ARG, "sq_lora_plan")
    if plan is None:
        plan = torch.empty(nbytes // 4, dtype=torch.int32, device=adapter.device)
    _shape(plan, torch.int32, (nbytes // 4,), "plan")
    _check(lib().sq_lora_plan(_ptr(adapter), M, n_adapters, _ptr(plan), _stream()),
           "sq_lora_plan")
    return plan


def _lora_weights(A: torch.Tensor, Bm: torch.Tensor, scale: torch.Tensor, plan: torch.Tensor,
                  M: int):
    _need(A, torch.bfloat16, "A")
    _need(Bm, torch.bfloat16, "B")
    if A.dim() != 3 or Bm.dim() != 3:
        raise ValueError("A must be [L, R, K] and B [L, N, R]")
    L, R, K = A.shape
    N = Bm.shape[1]
    _shape(A, torch.bfloat16, (L, R, K), "A")
    _shape(Bm, torch.bfloat16, (L, N, R), "B")
    _shape(scale, torch.float32, (L,), "scale")
    _here(A.device, B=Bm, scale=scale, plan=plan)
    _shape(plan, torch.int32, (sq_lora_plan_bytes(M, L) // 4,), "plan")
    return L, R, K, N


def sq_lora_forward(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                    plan: torch.Tensor, base: Optional[torch.Tensor],
                    y: Optional[torch.Tensor] = None, t: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """y = base + scale[a] B[a] (A[a] x) per row with adapter a -> (y, t).  base
    bf16 or fp32 [M, N] (None: zeros, bf16 unless y says otherwise); y may be base
    (in place); t fp32 [M, R] is kept for the backward pass (rows without an
    adapter are not written)."""
    _need(x, torch.bfloat16, "x")
    M, K, _ = _rows(x)
    L, R, Ka, N = _lora_weights(A, B, scale, plan, M)
    if Ka != K:
        raise ValueError(f"A has K = {Ka}, x has {K}")
    if y is None:
        y = torch.empty(M, N, dtype=torch.bfloat16 if base is None else base.dtype,
                        device=x.device)
    if t is None:
        t = torch.empty(M, R, dtype=torch.float32, device=x.device)
    out = _out_dtype(y, "y")
    _shape(y, y.dtype, (M, N), "y", contiguous=False)
    _shape(base, y.dtype, (M, N), "base", contiguous=False)
    _shape(t, torch.float32, (M, R), "t")
    if workspace is None:
        workspace = torch.empty(sq_lora_workspace_bytes(M, R, L, y.dtype), dtype=torch.uint8,
                                device=x.device)
    _need(workspace, torch.uint8, "workspace")
    _here(x.device, A=A, base=base, y=y, t=t, workspace=workspace)
    _check(lib().sq_lora_forward(_ptr(x), _ld(x), _ptr(A), _ptr(B), _ptr(scale), _ptr(plan),
                                 _ptr(base), 0 if base is None else _ld(base), _ptr(y), _ld(y),
                                 out, _ptr(t), _ptr(workspace), workspace.numel(), M, N, K, R, L,
                                 _stream()), "sq_lora_forward")
    return y, t


def sq_lora_workspace_bytes(M: int, R: int, n_adapters: int, dtype=torch.bfloat16) -> int:
    """Workspace bytes of sq_lora_forward (dtype of y) and sq_lora_backward (0:
    sizes out of range)."""
    return lib().sq_lora_workspace_bytes(M, R, n_adapters, _out_dtype(dtype, "dtype"))


def sq_lora_backward(dy: torch.Tensor, x: torch.Tensor, t: torch.Tensor, A: torch.Tensor,
                     B: torch.Tensor, scale: torch.Tensor, plan: torch.Tensor,
                     dx_base: Optional[torch.Tensor], dx: Optional[torch.Tensor] = None,
                     dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                     grad_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                     need_dx: bool = True, need_weights: bool = True):
    """Gradients of sq_lora_forward -> (dA, dB, dx): dA [L, R, K] and dB [L, N, R]
    of grad_dtype (bf16 or fp32; None without need_weights), dx = dx_base + the
    adapters' part (dx_base None: zeros; dx may be dx_base; None without need_dx)."""
    _need(dy, torch.bfloat16, "dy")
    _need(x, torch.bfloat16, "x")
    M, N, _ = _rows(dy)
    L, R, K, Nb = _lora_weights(A, B, scale, plan, M)
    if Nb != N:
        raise ValueError(f"B has N = {Nb}, dy has {N}")
    dev = dy.device
    if need_dx and dx is None:
        dx = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    if not need_dx:
        if dx is not None or dx_base is not None:
            raise ValueError("dx and dx_base are of no use without need_dx")
    if need_weights:
        if dA is None:
            dA = torch.empty(L, R, K, dtype=grad_dtype, device=dev)
        if dB is None:
            dB = torch.empty(L, N, R, dtype=grad_dtype, device=dev)
    elif dA is not None or dB is not None:
        raise ValueError("dA and dB are of no use without need_weights")
    out = _out_dtype(grad_dtype, "grad_dtype")
    if workspace is None:
        workspace = torch.empty(sq_lora_workspace_bytes(M, R, L, grad_dtype), dtype=torch.uint8,
                                device=dev)
    _need(workspace, torch.uint8, "workspace")
    _shape(x, torch.bfloat16, (M, K), "x", contiguous=False)
    _shape(t, torch.float32, (M, R), "t")
    _shape(dx_base, torch.bfloat16, (M, K), "dx_base", contiguous=False)
    _shape(dx, torch.bfloat16, (M, K), "dx", contiguous=False)
    _shape(dA, grad_dtype, (L, R, K), "dA")
    _shape(dB, grad_dtype, (L, N, R), "dB")
    _here(dev, x=x, t=t, A=A, dx_base=dx_base, dx=dx, dA=dA, dB=dB,
          workspace=workspace)
    _check(lib().sq_lora_backward(
        _ptr(dy), _ld(dy), _ptr(x), _ld(x), _ptr(t), _ptr(A), _ptr(B), _ptr(scale), _ptr(plan),
        _ptr(dx_base), 0 if dx_base is None else _ld(dx_base), _ptr(dx),
        0 if dx is None else _ld(dx), _ptr(dA), _ptr(dB), out, _ptr(workspace),
        workspace.numel(), M, N, K, R, L, _stream()), "sq_lora_backward")
    return dA, dB, dx


def sq_rope_frequencies(rot: int, base: float = 10000.0, scaling: int = SQ_ROPE_SCALE_NONE,
                        scale: float = 1.0, original_context: float = 0.0,
                        beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq, factor): fp32 CPU tensor [rot / 2] and the factor for the rotary
    calls; evaluated on the host in fp64."""
    if rot < 2 or rot % 2 or rot > 1024:
        raise SegQuantError(SQ_ERR_INVALID_ARG, "sq_rope_frequencies")
    inv_freq = torch.empty(rot // 2, dtype=torch.float32)
    factor = ctypes.c_float(1.0)
    _check(lib().sq_rope_frequencies(rot, base, scaling, scale, original_context, beta_fast,
                                     beta_slow, _ptr(inv_freq), ctypes.byref(factor)),
           "sq_rope_frequencies")
    return inv_freq, factor.value


def _rope(call: str, x, positions, inv_freq, head_dim, out, layout, axis_pairs, factor):
    dtype = _out_dtype(x, "x")
    M, cols, _ = _rows(x)
    _need(positions, torch.int32, "positions")
    _need(inv_freq, torch.float32, "inv_freq")
    if cols % head_dim != 0:
        raise ValueError(f"{cols} columns are no whole number of heads of {head_dim}")
    axes = 1 if axis_pairs is None else len(axis_pairs)
    if positions.dim() == 1 and axes == 1:
        positions = positions[:, None]
    _shape(positions, torch.int32, (M, axes), "positions")
    _shape(inv_freq, torch.float32, (inv_freq.numel(),), "inv_freq")
    if out is None:
        out = torch.empty(M, cols, dtype=x.dtype, device=x.device)
    _shape(out, x.dtype, (M, cols), "out", contiguous=False)
    _here(x.device, positions=positions, inv_freq=inv_freq, out=out)
    arr = None if axis_pairs is None else (ctypes.c_int32 * axes)(*[int(v) for v in axis_pairs])
    ldx = _ld(x)
    ldo = ldx if out.data_ptr() == x.data_ptr() and M <= 1 else _ld(out)
    _check(getattr(lib(), call)(_ptr(x), ldx, _ptr(out), ldo, dtype, _ptr(positions),
                                _ptr(inv_freq), arr, axes, float(factor), M, cols // head_dim,
                                head_dim, 2 * inv_freq.numel(), layout, _stream()), call)
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


def sq_group_norm_workspace_bytes(B: int, S: int, C: int, G: int) -> int:
    """Workspace bytes of the group norm calls (0: sizes out of range, or B = 0)."""
    return lib().sq_group_norm_workspace_bytes(B, S, C, G)


def _samples(t: Optional[torch.Tensor], shape, name: str):
    """A [B, S, C] bf16 tensor whose samples and rows lie at one row stride -> ld."""
    if t is None:
        return 0
    if t.dtype != torch.bfloat16 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be bf16 {list(shape)}, got {t.dtype} {list(t.shape)}")
    B, S, C = shape
    if t.numel() == 0:
        return (C + 7) // 8 * 8
    if S > 1:
        ld = t.stride(1)
    elif B > 1:
        ld = t.stride(0)
    else:
        ld = (C + 7) // 8 * 8
    if (C > 1 and t.stride(2) != 1) or (B > 1 and t.stride(0) != S * ld):
        raise ValueError(f"{name} must have unit channel stride and one row stride")
    return ld


def _gn_workspace(workspace, B, S, C, G, device):
    if workspace is None:
        return torch.empty(sq_group_norm_workspace_bytes(B, S, C, G), dtype=torch.uint8,
                           device=device)
    _need(workspace, torch.uint8, "workspace")
    return workspace


def sq_group_norm_forward(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor],
                          beta: Optional[torch.Tensor], eps: float = 1e-5,
                          act: int = SQ_ACT_NONE, y: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None):
    """y = act(group norm of x) over channels-last samples x bf16 [B, S, C] ->
    (y, mean, rstd); mean and rstd fp32 [B, groups] are kept for the backward
    pass.  gamma, beta bf16 [C] or None; y may be x (in place)."""
    _need(x, torch.bfloat16, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, S, C]")
    B, S, C = x.shape
    if y is None:
        y = torch.empty(B, S, C, dtype=torch.bfloat16, device=x.device)
    ldx, ldy = _samples(x, (B, S, C), "x"), _samples(y, (B, S, C), "y")
    _shape(gamma, torch.bfloat16, (C,), "gamma")
    _shape(beta, torch.bfloat16, (C,), "beta")
    stats = torch.empty(2, B, groups, dtype=torch.float32, device=x.device)
    workspace = _gn_workspace(workspace, B, S, C, groups, x.device)
    _here(x.device, gamma=gamma, beta=beta, y=y, workspace=workspace)
    _check(lib().sq_group_norm_forward(_ptr(x), ldx, B, S, C, groups, _ptr(gamma), _ptr(beta),
                                       float(eps), act, _ptr(y), ldy, _ptr(stats[0]),
                                       _ptr(stats[1]), _ptr(workspace), workspace.numel(),
                                       _stream()), "sq_group_norm_forward")
    return y, stats[0], stats[1]


def sq_group_norm_backward(dy: torch.Tensor, x: torch.Tensor, groups: int,
                           gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                           mean: torch.Tensor, rstd: torch.Tensor, act: int = SQ_ACT_NONE,
                           dx: Optional[torch.Tensor] = None, grad_dtype=torch.bfloat16,
                           workspace: Optional[torch.Tensor] = None, need_dx: bool = True):
    """Gradients of sq_group_norm_forward -> (dx, dgamma, dbeta); dgamma and dbeta
    [C] of grad_dtype (None where gamma or beta is None); dx may be dy."""
    _need(dy, torch.bfloat16, "dy")
    _need(x, torch.bfloat16, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, S, C]")
    B, S, C = x.shape
    if need_dx and dx is None:
        dx = torch.empty(B, S, C, dtype=torch.bfloat16, device=x.device)
    if not need_dx and dx is not None:
        raise ValueError("dx is of no use without need_dx")
    lddy, ldx = _samples(dy, (B, S, C), "dy"), _samples(x, (B, S, C), "x")
    lddx = _samples(dx, (B, S, C), "dx")
    _shape(gamma, torch.bfloat16, (C,), "gamma")
    _shape(beta, torch.bfloat16, (C,), "beta")
    _shape(mean, torch.float32, (B, groups), "mean")
    _shape(rstd, torch.float32, (B, groups), "rstd")
    out = _out_dtype(grad_dtype, "grad_dtype")
    dgamma = None if gamma is None else torch.empty(C, dtype=grad_dtype, device=x.device)
    dbeta = None if beta is None else torch.empty(C, dtype=grad_dtype, device=x.device)
    workspace = _gn_workspace(workspace, B, S, C, groups, x.device)
    _here(x.device, dy=dy, gamma=gamma, beta=beta, mean=mean, rstd=rstd, dx=dx,
          workspace=workspace)
    _check(lib().sq_group_norm_backward(_ptr(dy), lddy, _ptr(x), ldx, B, S, C, groups,
                                        _ptr(gamma), _ptr(beta), _ptr(mean), _ptr(rstd), act,
                                        _ptr(dx), lddx, _ptr(dgamma), _ptr(dbeta), out,
                                        _ptr(workspace), workspace.numel(), _stream()),
           "sq_group_norm_backward")
    return dx, dgamma, dbeta


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
    _need(dy, torch.bfloat16, "dy")
    _need(wq, torch.int8, "wq")
    if wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    M, N, _ = _rows(dy)
    K = wq.shape[1]
    _shape(wq, torch.int8, (N, K), "wq")
    _shape(s_w, torch.float32, (seg.S, N), "s_w")
    _shape(d, torch.float32, (seg.n_groups, K), "d")
    if dx is None:
        dx = torch.empty(M, K, dtype=torch.bfloat16, device=dy.device)
    _shape(dx, torch.bfloat16, (M, K), "dx", contiguous=False)
    if workspace is None:
        workspace = torch.empty(sq_input_grad_workspace_bytes(N, K), dtype=torch.uint8,
                                device=dy.device)
    _need(workspace, torch.uint8, "workspace")
    _here(dy.device, wq=wq, s_w=s_w, d=d, dx=dx, workspace=workspace)
    cs, keep = seg._c()
    _check(lib().sq_dualscale_seglinear_input_grad(
        _ptr(dy), _ld(dy), _ptr(wq), _ptr(s_w), _ptr(d), ctypes.byref(cs), _ptr(dx), _ld(dx), M,
        N, K, _ptr(workspace), workspace.numel(), _stream()),
        "sq_dualscale_seglinear_input_grad")
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
