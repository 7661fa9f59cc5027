"""Layer-level use of the library: one DualScale + SegLinear quantized linear,
its adapters and gradients, and what stands before an attention.

Offline (once): quantize the weight segment-wise and calibrate s+ / s- on a
calibration slice -- both on the GPU through the C ABI.  Online (per call):
quantize the activation into the stacked planes, then run the fused GEMM.
The quantized weight is frozen; adapters beside it are trained with the
explicit forward and backward calls below.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import binding as B


class Adapters:
    """The low-rank adapters of one layer: A bf16 [L][R][K], B bf16 [L][N][R],
    scale fp32 [L] (CUDA).  Adapter a adds scale[a] B[a] A[a] x to the layer's
    output of every row it is named for."""

    def __init__(self, A: torch.Tensor, B_: torch.Tensor, scale: torch.Tensor):
        if A.dim() != 3 or B_.dim() != 3 or A.shape[0] != B_.shape[0] or \
                A.shape[1] != B_.shape[2] or scale.shape != A.shape[:1]:
            raise ValueError("A must be [L, R, K], B [L, N, R] and scale [L]")
        self.A, self.B, self.scale = A, B_, scale

    def plan(self, ids: torch.Tensor) -> torch.Tensor:
        """The plan of a batch with adapter ids[m] (int32 [M]; -1: none) on row m;
        it serves every layer with as many adapters."""
        return B.sq_lora_plan(ids, self.A.shape[0])


class DualScaleSegLinear:
    """W8A8 DualScale linear with SegLinear segments.

    w      bf16 [N][K] nn.Linear weight (CUDA)
    bias   bf16 [N] or None
    d      fp32 [G][K] SmoothQuant divisor or None
    seg    binding.Segments
    x_cal  bf16 [rows][K] calibration activations
    weight_bits  8 (W8A8) or 4 (W4A8: weights kept packed, two codes per byte,
           and expanded into the int8 GEMM operand before every GEMM; several
           layers may share one operand buffer, `w_operand`, int8 [>= N*K])
    fp8    FP8 E4M3 codes for activations and weights (SQ_FLAG_FP8) instead of int8
    workspace  optional uint8 CUDA tensor from binding.gemm_workspace(): the GEMM
           then balances its last wave of tiles over all SMs (same results); layers
           run one after another on one stream may share one
    """

    def __init__(self, w: torch.Tensor, bias: Optional[torch.Tensor], d: Optional[torch.Tensor],
                 seg: B.Segments, x_cal: torch.Tensor, out_dtype=torch.bfloat16,
                 adaptive: bool = False, asymmetry_threshold: float = 2.0,
                 weight_bits: int = 8, w_operand: Optional[torch.Tensor] = None,
                 fp8: bool = False, workspace: Optional[torch.Tensor] = None):
        if weight_bits not in (8, 4):
            raise ValueError("weight_bits must be 8 or 4")
        if fp8 and weight_bits == 4:
            raise ValueError("FP8 codes and W4 weights do not combine")
        self.N, self.K = w.shape
        self.weight_bits = weight_bits
        self.workspace = workspace
        self.fp8 = fp8
        if weight_bits == 4:
            seg = B.Segments(seg.mode, seg.offsets, seg.n_groups, seg.flags | B.SQ_FLAG_W4)
        if fp8:
            seg = B.Segments(seg.mode, seg.offsets, seg.n_groups, seg.flags | B.SQ_FLAG_FP8)
        self.seg = seg
        self.G, self.S = seg.n_groups, seg.S
        self.d = d
        self.bias = bias
        self.out_dtype = out_dtype
        dev = w.device
        self.s_w = torch.empty(self.S, self.N, dtype=torch.float32, device=dev)
        if weight_bits == 4:
            self.wq4 = torch.empty(self.N, self.K // 2, dtype=torch.uint8, device=dev)
            B.sq_quantize_weight_w4(w, d, seg, self.wq4, self.s_w)
            if w_operand is None:
                w_operand = torch.empty(self.N * self.K, dtype=torch.int8, device=dev)
            if w_operand.numel() < self.N * self.K or w_operand.dtype != torch.int8:
                raise ValueError("w_operand must be int8 with at least N*K elements")
            self.wq = w_operand.view(-1)[: self.N * self.K].view(self.N, self.K)
        else:
            self.wq4 = None
            self.wq = torch.empty(self.N, self.K, dtype=torch.int8, device=dev)
            B.sq_quantize_weight_seg(w, d, seg, self.wq, self.s_w)
        self.s_act = torch.empty(self.G, self.S, 2, dtype=torch.float32, device=dev)
        B.sq_calibrate_act(x_cal, d, seg, self.s_act)
        if adaptive and not seg.flags & B.SQ_FLAG_SINGLE_SCALE:
            # Adaptive DualScale (the library's policy call): keep the two steps
            # only where the calibrated sides differ by at least
            # `asymmetry_threshold` in some group and K-segment; otherwise
            # switch the layer to one symmetric step.
            if B.sq_choose_single_scale(self.s_act, fp8=fp8, threshold=asymmetry_threshold):
                self.seg = B.Segments(seg.mode, seg.offsets, seg.n_groups,
                                      seg.flags | B.SQ_FLAG_SINGLE_SCALE)
                B.sq_calibrate_act(x_cal, d, self.seg, self.s_act)
        self.single_scale = bool(self.seg.flags & B.SQ_FLAG_SINGLE_SCALE)
        # With SmoothQuant divisors: the channels whose codes may skip both
        # quotient corrections (same codes; sq_quantize_act_plan).
        self.plan = (B.sq_quantize_act_plan(d, self.s_act, self.seg)
                     if d is not None and not fp8 else None)
        self._planes = None

    def planes_for(self, M: int, device) -> torch.Tensor:
        if self._planes is None or self._planes.shape[2] != M:
            self._planes = torch.empty(self.G, self.seg.P, M, self.K, dtype=torch.int8,
                                       device=device)
        return self._planes

    def quantize(self, x: torch.Tensor, planes: Optional[torch.Tensor] = None) -> torch.Tensor:
        if planes is None:
            planes = self.planes_for(x.shape[0], x.device)
        return B.sq_quantize_act(x, self.d, self.s_act, self.seg, planes, plan=self.plan)

    def gemm(self, planes: torch.Tensor, y: Optional[torch.Tensor] = None) -> torch.Tensor:
        M = planes.shape[2]
        if y is None:
            y = torch.empty(M, self.N, dtype=self.out_dtype, device=planes.device)
        if self.wq4 is not None:
            B.sq_unpack_weight_w4(self.wq4, self.wq)
        return B.sq_dualscale_seglinear_gemm(planes, self.wq, self.s_w, self.s_act, self.bias,
                                             y, self.seg, workspace=self.workspace)

    def gemm_gelu_quant(self, planes: torch.Tensor, nxt: "DualScaleSegLinear",
                        planes_next: Optional[torch.Tensor] = None) -> torch.Tensor:
        """This layer's GEMM fused with the next layer's input: returns nxt's
        activation planes of bf16(gelu(bf16(y))) (an FFN's fc1 feeding fc2),
        computed in this GEMM's epilogue with nxt's calibrated steps.  This
        layer: one K-segment; nxt: one group and K-segment, no divisor."""
        if nxt.d is not None or nxt.seg.mode != B.SQ_SEG_NONE:
            raise ValueError("the next layer must have one segment and no SmoothQuant divisor")
        M = planes.shape[2]
        if planes_next is None:
            planes_next = torch.empty(1, nxt.seg.P, M, nxt.K, dtype=torch.int8,
                                      device=planes.device)
        if self.wq4 is not None:
            B.sq_unpack_weight_w4(self.wq4, self.wq)
        return B.sq_dualscale_seglinear_gemm_gelu_quant(planes, self.wq, self.s_w, self.s_act,
                                                        self.bias, self.seg,
                                                        nxt.s_act.reshape(2), planes_next,
                                                        single_next=nxt.seg.P == 1)

    def __call__(self, x: torch.Tensor, y: Optional[torch.Tensor] = None) -> torch.Tensor:
        return self.gemm(self.quantize(x), y)

    def adapted(self, x: torch.Tensor, adapters: Adapters, plan: torch.Tensor,
                y: Optional[torch.Tensor] = None):
        """(y, t): the layer's output with its rows' adapters added, in place on
        the GEMM's output, and t [M, R] for adapted_backward."""
        y = self(x, y)
        return B.sq_lora_forward(x, adapters.A, adapters.B, adapters.scale, plan, y, y=y)

    def input_grad(self, dy: torch.Tensor, dx: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dL/dx of the frozen layer from dy bf16 [M, N], straight through the
        activation quantizer."""
        if self.wq4 is not None:
            B.sq_unpack_weight_w4(self.wq4, self.wq)
        return B.sq_dualscale_seglinear_input_grad(dy, self.wq, self.s_w, self.d, self.seg, dx=dx,
                                                   workspace=workspace)

    def adapted_backward(self, dy: torch.Tensor, x: torch.Tensor, t: torch.Tensor,
                         adapters: Adapters, plan: torch.Tensor, grad_dtype=torch.bfloat16,
                         need_dx: bool = True):
        """(dA, dB, dx) of adapted(); x is its input and t its second result.  dx
        (None without need_dx) joins the frozen layer's part and the adapters'."""
        dx = self.input_grad(dy) if need_dx else None
        return B.sq_lora_backward(dy, x, t, adapters.A, adapters.B, adapters.scale, plan, dx,
                                  dx=dx, grad_dtype=grad_dtype, need_dx=need_dx)


class AttentionGrads(NamedTuple):
    x: torch.Tensor                 # bf16 [B, S, C]
    gamma: Optional[torch.Tensor]   # [C]
    beta: Optional[torch.Tensor]
    A: Optional[torch.Tensor]       # as the adapters
    B: Optional[torch.Tensor]


class AttentionInput:
    """From features to q|k|v: an optional channels-last group norm with its
    activation, the quantized projection with its rows' adapters, and rotary
    positions on the q and k columns, in place.

    qkv       DualScaleSegLinear with bf16 output, columns q | k | v
    head_dim  columns of a head
    rotated_heads  heads that turn: q's and k's, the first columns of the output
    inv_freq  fp32 CUDA [rot / 2], with `factor` from binding.sq_rope_frequencies
    layout, axis_pairs  as in binding.sq_rope_forward
    groups    groups of the norm (0: no norm); gamma, beta, eps, act as in
              binding.sq_group_norm_forward
    """

    def __init__(self, qkv: DualScaleSegLinear, head_dim: int, rotated_heads: int,
                 inv_freq: torch.Tensor, factor: float = 1.0,
                 layout: int = B.SQ_ROPE_INTERLEAVED, axis_pairs: Optional[Sequence[int]] = None,
                 groups: int = 0, gamma: Optional[torch.Tensor] = None,
                 beta: Optional[torch.Tensor] = None, eps: float = 1e-5,
                 act: int = B.SQ_ACT_NONE):
        if qkv.out_dtype != torch.bfloat16:
            raise ValueError("the projection must write bf16")
        if head_dim < 1 or rotated_heads < 1 or rotated_heads * head_dim > qkv.N:
            raise ValueError("the rotated heads must lie within the projection's output")
        if groups == 0 and (gamma is not None or beta is not None or act != B.SQ_ACT_NONE):
            raise ValueError("gamma, beta and act belong to a norm (groups > 0)")
        self.qkv, self.head_dim, self.turned = qkv, head_dim, rotated_heads * head_dim
        self.inv_freq, self.factor = inv_freq, factor
        self.layout, self.axis_pairs = layout, axis_pairs
        self.groups, self.gamma, self.beta, self.eps, self.act = groups, gamma, beta, eps, act

    def _rope(self, call, x, positions, out):
        return call(x, positions, self.inv_freq, self.head_dim, out, layout=self.layout,
                    axis_pairs=self.axis_pairs, factor=self.factor)

    def forward(self, x: torch.Tensor, positions: torch.Tensor,
                adapters: Optional[Adapters] = None, plan: Optional[torch.Tensor] = None):
        """x bf16 [B, S, C] -> (q|k|v bf16 [B * S, N], saved); positions int32
        [B * S] or [B * S, axes]; adapters and plan (of the B * S rows) together."""
        if (adapters is None) != (plan is None):
            raise ValueError("adapters and plan come together")
        mean = rstd = t = None
        h = x
        if self.groups:
            h, mean, rstd = B.sq_group_norm_forward(x, self.groups, self.gamma, self.beta,
                                                    eps=self.eps, act=self.act)
        h = h.reshape(-1, x.shape[2])
        if adapters is None:
            y = self.qkv(h)
        else:
            y, t = self.qkv.adapted(h, adapters, plan)
        qk = y[:, :self.turned]
        self._rope(B.sq_rope_forward, qk, positions, qk)
        return y, (x, h, mean, rstd, t, positions, adapters, plan)

    __call__ = forward

    def backward(self, dy: torch.Tensor, saved, grad_dtype=torch.bfloat16) -> AttentionGrads:
        """The gradients of forward() from dy bf16 [B * S, N], whose q and k columns
        are turned back in place."""
        x, h, mean, rstd, t, positions, adapters, plan = saved
        qk = dy[:, :self.turned]
        self._rope(B.sq_rope_backward, qk, positions, qk)
        dA = dB = dgamma = dbeta = None
        if adapters is None:
            dx = self.qkv.input_grad(dy)
        else:
            dA, dB, dx = self.qkv.adapted_backward(dy, h, t, adapters, plan, grad_dtype)
        dx = dx.view(x.shape)
        if self.groups:
            dx, dgamma, dbeta = B.sq_group_norm_backward(dx, x, self.groups, self.gamma, self.beta,
                                                         mean, rstd, act=self.act, dx=dx,
                                                         grad_dtype=grad_dtype)
        return AttentionGrads(dx, dgamma, dbeta, dA, dB)
