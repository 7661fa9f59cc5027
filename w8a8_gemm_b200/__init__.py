"""SegQuant DualScale + SegLinear W8A8 linear layer for NVIDIA B200 (sm_100a).

The computation lives in libsegquant.so (C ABI: include/segquant.h); this
package holds its build script, a thin ctypes binding with the same entry-point
names, layer-level wrappers (the quantized linear, its adapters and gradients,
the input side of an attention), and the seeded synthetic workloads.
Importing the package never loads CUDA; the first library call does, and fails
loudly if the library has not been built.
"""
from .binding import (HostPipeline, SQ_ACT_GELU, SQ_ACT_NONE, SQ_ACT_SILU, SQ_FLAG_FP8,
                      SQ_FLAG_SINGLE_SCALE, SQ_FLAG_W4, SQ_OUT_BF16, SQ_OUT_F32, SQ_ROPE_HALF,
                      SQ_ROPE_INTERLEAVED, SQ_ROPE_SCALE_LINEAR, SQ_ROPE_SCALE_NONE,
                      SQ_ROPE_SCALE_NTK, SQ_ROPE_SCALE_YARN, SQ_SEG_INPUT, SQ_SEG_NONE,
                      SQ_SEG_OUTPUT, SegQuantError, Segments, sq_calibrate_act,
                      sq_choose_single_scale, sq_debug_gemm_s32, sq_dualscale_seglinear_gemm,
                      sq_dualscale_seglinear_gemm_gelu_quant, sq_dualscale_seglinear_host,
                      sq_dualscale_seglinear_host_noalloc, sq_dualscale_seglinear_input_grad,
                      sq_get_device_status, sq_group_norm_backward, sq_group_norm_forward,
                      sq_group_norm_workspace_bytes, sq_input_grad_workspace_bytes,
                      sq_lora_backward, sq_lora_forward, sq_lora_plan, sq_lora_plan_bytes,
                      sq_lora_workspace_bytes, sq_quantize_act, sq_quantize_weight_seg,
                      sq_quantize_weight_w4, sq_rope_backward, sq_rope_forward,
                      sq_rope_frequencies, sq_unpack_weight_w4, sq_version)

__all__ = ["HostPipeline", "SQ_ACT_GELU", "SQ_ACT_NONE", "SQ_ACT_SILU", "SQ_FLAG_FP8",
           "SQ_FLAG_SINGLE_SCALE", "SQ_FLAG_W4", "SQ_OUT_BF16", "SQ_OUT_F32", "SQ_ROPE_HALF",
           "SQ_ROPE_INTERLEAVED", "SQ_ROPE_SCALE_LINEAR", "SQ_ROPE_SCALE_NONE",
           "SQ_ROPE_SCALE_NTK", "SQ_ROPE_SCALE_YARN", "SQ_SEG_INPUT", "SQ_SEG_NONE",
           "SQ_SEG_OUTPUT", "SegQuantError", "Segments", "sq_calibrate_act",
           "sq_choose_single_scale", "sq_debug_gemm_s32", "sq_dualscale_seglinear_gemm",
           "sq_dualscale_seglinear_gemm_gelu_quant", "sq_dualscale_seglinear_host",
           "sq_dualscale_seglinear_host_noalloc", "sq_dualscale_seglinear_input_grad",
           "sq_get_device_status", "sq_group_norm_backward", "sq_group_norm_forward",
           "sq_group_norm_workspace_bytes", "sq_input_grad_workspace_bytes", "sq_lora_backward",
           "sq_lora_forward", "sq_lora_plan", "sq_lora_plan_bytes", "sq_lora_workspace_bytes",
           "sq_quantize_act", "sq_quantize_weight_seg", "sq_quantize_weight_w4",
           "sq_rope_backward", "sq_rope_forward", "sq_rope_frequencies", "sq_unpack_weight_w4",
           "sq_version"]
