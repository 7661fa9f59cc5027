// sq_internal.h -- declarations shared by the library's own translation units
// (kernels and the C-ABI layer).  Not installed; not used by anything else.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/segquant.h"

namespace sq {

// Segment table as the kernels see it (passed by value as a kernel argument).
struct SegParams {
  int32_t mode;   // sq_seg_mode
  int32_t n_seg;  // segments
  int32_t G;      // activation groups
  int32_t S;      // K-segments (n_seg in input mode, else 1)
  int32_t P;      // activation planes per group: 2 (DualScale) or 1 (single scale)
  int32_t w4;     // 1: the weight operand holds 16 q of W4A8 codes q (SQ_FLAG_W4)
  int32_t fp8;    // 1: codes are FP8 E4M3 bit patterns (SQ_FLAG_FP8)
  int32_t off[SQ_MAX_SEGMENTS + 1];
};

// Guard of a plain global store: `ok` is the test of the store's index against
// its buffer's logical extent.  In the bounds-checked debug build
// (SQ_DEBUG_BOUNDS) a failed test records SQ_ERR_DEVICE_BOUNDS in `status`
// (first report wins) and the caller skips the store; in the release build the
// guard is always true and costs nothing.
__device__ __forceinline__ bool store_ok(int *status, bool ok) {
#ifdef SQ_DEBUG_BOUNDS
  if (!ok) atomicCAS(status, 0, static_cast<int>(SQ_ERR_DEVICE_BOUNDS));
  return ok;
#else
  (void)status;
  (void)ok;
  return true;
#endif
}

// Index i with off[i] <= p < off[i + 1] (tables are short: a linear scan).
__host__ __device__ inline int seg_index(const int32_t *off, int n_seg, int64_t p) {
  int i = 0;
  while (i + 1 < n_seg && p >= off[i + 1]) ++i;
  return i;
}

// ---- launchers (quant.cu) --------------------------------------------------
cudaError_t launch_calibrate_act(const uint16_t *x, int64_t M, int64_t K, int64_t ldx,
                                 const float *d, const SegParams &seg, float *s_act,
                                 int *status, cudaStream_t stream);
sq_status launch_quantize_act(const uint16_t *x, int64_t M, int64_t K, int64_t ldx,
                              const float *d, const float *s_act, const SegParams &seg,
                              int8_t *planes, const uint32_t *plan, int *status,
                              cudaStream_t stream);
// Quantize plan: bits [G][ceil(K/32)] (see quant_plan_kernel).
cudaError_t launch_quantize_plan(const float *d, int64_t K, const float *s_act,
                                 const SegParams &seg, uint32_t *plan, int *status,
                                 cudaStream_t stream);
cudaError_t launch_quantize_weight(const uint16_t *w, int64_t N, int64_t K, const float *d,
                                   const SegParams &seg, int8_t *wq, float *s_w, int *status,
                                   cudaStream_t stream);
cudaError_t launch_quantize_weight_w4(const uint16_t *w, int64_t N, int64_t K, const float *d,
                                      const SegParams &seg, uint8_t *wq4, float *s_w,
                                      int *status, cudaStream_t stream);
cudaError_t launch_unpack_w4(const uint8_t *wq4, int64_t N, int64_t K, int8_t *wq, int *status,
                             cudaStream_t stream);

// ---- launcher (gemm.cu) ----------------------------------------------------
// OUT_PLANES: the next layer's int8 activation planes, from bf16(gelu(bf16(y)))
// (the fused producer of an FFN's second linear).
enum OutKind { OUT_BF16 = 0, OUT_F32 = 1, OUT_S32 = 2, OUT_PLANES = 3 };

struct GemmRequest {
  const int8_t *planes;
  const int8_t *wq;
  const float *s_w;
  const float *s_act;
  const uint16_t *bias;
  void *y;
  int64_t ldy;
  int out_kind;
  int64_t M, N, K;
  SegParams seg;
  int *status;  // device error word
  // OUT_PLANES: the next layer's steps {s+, s-} (fp32 [2], device) and its
  // planes per group (2 DualScale, 1 single scale); y is int8 [p_next][M][N].
  const float *s_next = nullptr;
  int p_next = 0;
  // Optional workspace for the split last wave (zero-filled before its first
  // use; every call leaves its flags at zero): nullptr = whole tiles only.
  void *workspace = nullptr;
  size_t workspace_bytes = 0;
};

sq_status launch_gemm(const GemmRequest &req, cudaStream_t stream);
// Workspace bytes that let any one-segment GEMM split its last wave on the
// current device.
size_t gemm_workspace_bytes();

// ---- low-rank adapters (lora.cu) ---------------------------------------------
// Rows of one tile of the plan.
#define SQ_LORA_TILE_ROWS 128

struct LoraRequest {
  const uint16_t *x, *dy, *A, *B;
  const float *scale;
  const int32_t *plan;
  const void *base;      // forward: y's, backward: dx's; nullptr: zeros
  void *y;               // forward
  uint16_t *dx;          // backward, may be nullptr
  void *dA, *dB;         // backward, both or neither
  float *t;              // [M][R]
  void *workspace;
  int64_t ldx, lddy, ld_base, ldy, lddx;
  int64_t M, N, K;
  int32_t R, L;
  bool f32;              // forward: base and y are fp32; backward: dA and dB are
  int *status;
};
size_t lora_plan_words(int64_t M, int32_t L);
// Of the backward call; the forward call uses half of it.
size_t lora_workspace_bytes(int64_t M, int32_t R, int32_t L, bool f32);
cudaError_t launch_lora_plan(const int32_t *adapter, int64_t M, int32_t L, int32_t *plan,
                             int *status, cudaStream_t stream);
cudaError_t launch_lora_forward(const LoraRequest &q, cudaStream_t stream);
cudaError_t launch_lora_backward(const LoraRequest &q, cudaStream_t stream);

// ---- rotary positions (rope.cu) ----------------------------------------------
struct RopeArgs {
  const void *x;
  int64_t ldx;
  void *out;
  int64_t ldo;
  const int32_t *positions;  // [M][axes]
  const float *inv_freq;     // [rot / 2]
  int64_t M;
  int32_t H, D, rot, axes;
  int32_t axis_end[SQ_ROPE_MAX_AXES];  // pairs before the end of each axis
  float factor, sign;
  int32_t rows_per_block;    // set by the launcher
  int *status;
};
cudaError_t launch_rope(const RopeArgs &p, bool half, bool f32, cudaStream_t stream);

// ---- group norm (group_norm.cu) ----------------------------------------------
constexpr int kGroupNormMaxC = 8192, kGroupNormMaxG = 1024;
struct GroupNormArgs {
  const uint16_t *x, *dy;
  uint16_t *y, *dx;
  int64_t ldx, lddy, ldy, lddx;
  const uint16_t *gamma, *beta;  // nullptr: 1 and 0
  float *mean, *rstd;            // [B][G]; forward writes, backward reads
  void *dgamma, *dbeta;          // [C], may be nullptr
  int64_t S;
  int32_t B, C, G;
  float eps;
  // set by the launcher
  int32_t rows_per_chunk, chunks, rows2, chunks2, slice, slices, grad_blocks;
  float2 *part, *chan_part;
  int *status;
};
size_t group_norm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G);
cudaError_t launch_group_norm_forward(GroupNormArgs p, void *workspace, int act,
                                      cudaStream_t stream);
cudaError_t launch_group_norm_backward(GroupNormArgs p, void *workspace, int act, bool gf32,
                                       cudaStream_t stream);

// ---- input gradient of a quantized linear (input_grad.cu) ----------------------
struct InputGradRequest {
  const uint16_t *dy;
  int64_t lddy;
  const int8_t *wq;
  const float *s_w, *d;
  SegParams seg;
  uint16_t *dx;
  int64_t lddx;
  void *workspace;
  int64_t M, N, K;
  int *status;
};
size_t input_grad_workspace_bytes(int64_t N, int64_t K);
sq_status launch_input_grad(const InputGradRequest &r, cudaStream_t stream);

// ---- test-only probes (probe.cu) -------------------------------------------
cudaError_t launch_timeout_probe(uint32_t limit_us, int *status, cudaStream_t stream);
// Debug build only: one checked store to element n of a buffer said to hold n.
cudaError_t launch_bounds_probe(int32_t *buf, int64_t n, int *status, cudaStream_t stream);

// Host-side validation of a quantize / GEMM call without launching anything
// (the checks of sq_quantize_act and sq_dualscale_seglinear_gemm).
sq_status validate_quantize_act(const void *x, int64_t M, int64_t K, int64_t ldx, const float *d,
                                const float *s_act, const sq_segments *seg, int8_t *planes);
sq_status validate_gemm(const int8_t *planes, const int8_t *wq, const float *s_w,
                        const float *s_act, const void *bias, void *y, int out_kind, int64_t M,
                        int64_t N, int64_t K, int64_t ldy, const sq_segments *seg);

// Device address of the library's error word on the current device.
int *device_status_word();

// SMs of the current device.
int sm_count();

// SQ_OK if the current device is an sm_100.
sq_status check_device();

// Validates a segment table.  extent_n < 0 means N is not known to the call
// (activation-side calls), in which case the output offsets end is not checked.
sq_status parse_segments(const sq_segments *seg, int64_t K, int64_t extent_n, SegParams *out);

// cuTensorMapEncodeTiled, resolved through the runtime (no link-time libcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();  // nullptr if the driver lacks it

}  // namespace sq
