// api_ops.cu -- the C ABI of the operators around the quantized linear (low-rank
// adapters, rotary positions, group norm, input gradient): argument validation
// on the host and dispatch to their kernels.  Nothing here allocates.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "spans.h"
#include "sq_internal.h"

namespace sq {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 44;  // more fit no device
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int32_t kMaxAdapters = 1024;
constexpr int32_t kMaxRank = 128;

#define SQ_TRY(expr)               \
  do {                             \
    const sq_status _s = (expr);   \
    if (_s != SQ_OK) return _s;    \
  } while (0)

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
sq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SQ_OK : SQ_ERR_CUDA; }
cudaStream_t cs(sq_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// A row-major buffer of `rows` rows of `cols` elements: leading dimension and,
// with rows, presence and alignment.
sq_status check_rows(const void *p, int64_t rows, int64_t cols, int64_t ld) {
  if (ld < cols) return SQ_ERR_INVALID_ARG;
  if (rows > 0 && ld > kMaxElems / rows) return SQ_ERR_INVALID_ARG;
  if (ld % 8 != 0) return SQ_ERR_ALIGNMENT;
  if (rows > 0 && p == nullptr) return SQ_ERR_INVALID_ARG;
  return aligned(p, 16) ? SQ_OK : SQ_ERR_ALIGNMENT;
}

// The device and its error word.
sq_status device_word(int **status) {
  SQ_TRY(check_device());
  *status = device_status_word();
  return *status != nullptr ? SQ_OK : SQ_ERR_CUDA;
}

bool lora_sizes_ok(int64_t M, int32_t L) {
  return M >= 0 && M <= kMaxRows && L >= 1 && L <= kMaxAdapters;
}

sq_status check_lora(int64_t M, int64_t N, int64_t K, int32_t R, int32_t L, const void *A,
                     const void *B, const float *scale, const int32_t *plan) {
  if (!lora_sizes_ok(M, L) || N < 8 || N > kMaxCols || K < 8 || K > kMaxCols)
    return SQ_ERR_INVALID_ARG;
  if (R < 8 || R > kMaxRank) return R < 1 ? SQ_ERR_INVALID_ARG : SQ_ERR_UNSUPPORTED;
  if (N % 8 != 0 || K % 8 != 0 || R % 8 != 0) return SQ_ERR_ALIGNMENT;
  if (A == nullptr || B == nullptr || scale == nullptr || plan == nullptr)
    return SQ_ERR_INVALID_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(scale, 4) || !aligned(plan, 16))
    return SQ_ERR_ALIGNMENT;
  return SQ_OK;
}

// The inputs of an adapter call that are single runs of bytes.
struct LoraSpans {
  Span A, B, scale, plan;
  LoraSpans(int64_t M, int64_t N, int64_t K, int64_t R, int32_t L, const void *a, const void *b,
            const void *s, const void *p)
      : A(a, L * R * K * 2), B(b, L * R * N * 2), scale(s, L * int64_t(4)),
        plan(p, static_cast<int64_t>(lora_plan_words(M, L)) * 4) {}
};

sq_status rope_common(const void *x, int64_t ldx, void *out, int64_t ldo, sq_out_dtype dtype,
                      const int32_t *positions, const float *inv_freq, const int32_t *axis_pairs,
                      int32_t n_axes, float factor, int64_t M, int32_t H, int32_t D, int32_t rot,
                      sq_rope_layout layout, float sign, sq_stream_t stream) {
  if (dtype != SQ_OUT_BF16 && dtype != SQ_OUT_F32) return SQ_ERR_INVALID_ARG;
  if (layout != SQ_ROPE_INTERLEAVED && layout != SQ_ROPE_HALF) return SQ_ERR_INVALID_ARG;
  if (M < 0 || M > INT32_MAX || H < 1 || D < 8 || D > 1024 || rot < 2 || rot > D || rot % 2 != 0)
    return SQ_ERR_INVALID_ARG;
  const int64_t cols = static_cast<int64_t>(H) * D;
  if (cols > kMaxCols || !isfinite(factor)) return SQ_ERR_INVALID_ARG;
  if (D % 8 != 0) return SQ_ERR_ALIGNMENT;
  if (n_axes < 1 || n_axes > SQ_ROPE_MAX_AXES || (axis_pairs == nullptr && n_axes != 1))
    return SQ_ERR_INVALID_ARG;
  RopeArgs p = {};
  int64_t pairs = 0;
  for (int32_t a = 0; a < n_axes; ++a) {
    const int32_t n = axis_pairs ? axis_pairs[a] : rot / 2;
    if (n < 0) return SQ_ERR_INVALID_ARG;
    pairs += n;
    if (pairs > rot / 2) return SQ_ERR_INVALID_ARG;
    p.axis_end[a] = static_cast<int32_t>(pairs);
  }
  if (pairs != rot / 2) return SQ_ERR_INVALID_ARG;
  SQ_TRY(check_rows(x, M, cols, ldx));
  SQ_TRY(check_rows(out, M, cols, ldo));
  if (M == 0) return SQ_OK;
  if (positions == nullptr || inv_freq == nullptr) return SQ_ERR_INVALID_ARG;
  if (x == out && ldx != ldo) return SQ_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return SQ_ERR_ALIGNMENT;
  const int64_t e = dtype == SQ_OUT_F32 ? 4 : 2;
  const Span from(x, M, cols * e, ldx * e), to(out, M, cols * e, ldo * e);
  if ((x != out && overlap(to, from)) ||
      overlaps_any(to, Span(positions, M * n_axes * 4), Span(inv_freq, rot / 2 * 4)))
    return SQ_ERR_INVALID_ARG;
  SQ_TRY(device_word(&p.status));
  p.x = x;
  p.ldx = ldx;
  p.out = out;
  p.ldo = ldo;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.M = M;
  p.H = H;
  p.D = D;
  p.rot = rot;
  p.axes = n_axes;
  p.factor = factor;
  p.sign = sign;
  return from_cuda(launch_rope(p, layout == SQ_ROPE_HALF, dtype == SQ_OUT_F32, cs(stream)));
}

bool group_norm_sizes_ok(int64_t B, int64_t S, int64_t C, int64_t G) {
  return B >= 0 && B <= 65535 && S >= 1 && S <= kMaxRows && C >= 8 && C <= kGroupNormMaxC &&
         C % 8 == 0 && G >= 1 && G <= kGroupNormMaxG && C % G == 0;
}

sq_status check_group_norm(int64_t B, int64_t S, int64_t C, int64_t G, const void *gamma,
                           const void *beta, int act, const float *mean, const float *rstd,
                           void *workspace, size_t workspace_bytes) {
  if (!group_norm_sizes_ok(B, S, C, G)) return SQ_ERR_INVALID_ARG;
  if (act < SQ_ACT_NONE || act > SQ_ACT_GELU) return SQ_ERR_INVALID_ARG;
  if (B == 0) return SQ_OK;
  if (mean == nullptr || rstd == nullptr || workspace == nullptr) return SQ_ERR_INVALID_ARG;
  if (workspace_bytes < group_norm_workspace_bytes(B, S, C, G)) return SQ_ERR_INVALID_ARG;
  if ((gamma && !aligned(gamma, 2)) || (beta && !aligned(beta, 2)) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(workspace, 16))
    return SQ_ERR_ALIGNMENT;
  return SQ_OK;
}

GroupNormArgs group_norm_args(const void *x, int64_t ldx, int64_t B, int64_t S, int64_t C,
                              int64_t G, const void *gamma, const void *beta, float *mean,
                              float *rstd, int *status) {
  GroupNormArgs p = {};
  p.x = static_cast<const uint16_t *>(x);
  p.ldx = ldx;
  p.B = static_cast<int32_t>(B);
  p.S = S;
  p.C = static_cast<int32_t>(C);
  p.G = static_cast<int32_t>(G);
  p.gamma = static_cast<const uint16_t *>(gamma);
  p.beta = static_cast<const uint16_t *>(beta);
  p.mean = mean;
  p.rstd = rstd;
  p.status = status;
  return p;
}

}  // namespace
}  // namespace sq

using namespace sq;

extern "C" {

size_t sq_lora_plan_bytes(int64_t M, int32_t n_adapters) {
  return lora_sizes_ok(M, n_adapters) ? lora_plan_words(M, n_adapters) * sizeof(int32_t) : 0;
}

size_t sq_lora_workspace_bytes(int64_t M, int32_t R, int32_t n_adapters,
                               sq_out_dtype grad_dtype) {
  if (!lora_sizes_ok(M, n_adapters) || R < 8 || R > kMaxRank || R % 8 != 0) return 0;
  if (grad_dtype != SQ_OUT_BF16 && grad_dtype != SQ_OUT_F32) return 0;
  return lora_workspace_bytes(M, R, n_adapters, grad_dtype == SQ_OUT_F32);
}

sq_status sq_lora_plan(const int32_t *adapter, int64_t M, int32_t n_adapters, int32_t *plan,
                       sq_stream_t stream) {
  if (!lora_sizes_ok(M, n_adapters)) return SQ_ERR_INVALID_ARG;
  if ((M > 0 && adapter == nullptr) || plan == nullptr) return SQ_ERR_INVALID_ARG;
  if (!aligned(adapter, 4) || !aligned(plan, 16)) return SQ_ERR_ALIGNMENT;
  if (overlap(Span(plan, lora_plan_words(M, n_adapters) * 4), Span(adapter, M * 4)))
    return SQ_ERR_INVALID_ARG;
  int *status = nullptr;
  SQ_TRY(device_word(&status));
  return from_cuda(launch_lora_plan(adapter, M, n_adapters, plan, status, cs(stream)));
}

sq_status sq_lora_forward(const void *x, int64_t ldx, const void *A, const void *B,
                          const float *scale, const int32_t *plan, const void *base,
                          int64_t ldbase, void *y, int64_t ldy, sq_out_dtype out_dtype, float *t,
                          void *workspace, size_t workspace_bytes, int64_t M, int64_t N,
                          int64_t K, int32_t R, int32_t n_adapters, sq_stream_t stream) {
  if (out_dtype != SQ_OUT_BF16 && out_dtype != SQ_OUT_F32) return SQ_ERR_INVALID_ARG;
  SQ_TRY(check_lora(M, N, K, R, n_adapters, A, B, scale, plan));
  SQ_TRY(check_rows(x, M, K, ldx));
  SQ_TRY(check_rows(y, M, N, ldy));
  if (base != nullptr) SQ_TRY(check_rows(base, M, N, ldbase));
  if (M == 0) return SQ_OK;
  const bool f32 = out_dtype == SQ_OUT_F32;
  if (t == nullptr || y == x || (base == y && ldbase != ldy)) return SQ_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < lora_workspace_bytes(M, R, n_adapters, f32))
    return SQ_ERR_INVALID_ARG;
  if (!aligned(t, 16) || !aligned(workspace, 16)) return SQ_ERR_ALIGNMENT;
  const int64_t e = f32 ? 4 : 2;
  const LoraSpans in(M, N, K, R, n_adapters, A, B, scale, plan);
  const Span sx(x, M, K * 2, ldx * 2), sy(y, M, N * e, ldy * e), st(t, M * R * 4),
      sw(workspace, lora_workspace_bytes(M, R, n_adapters, f32)),
      sb(base, base ? M : 0, N * e, ldbase * e);
  if ((base != y && overlap(sy, sb)) || overlaps_any(sy, sx, in.A, in.B, in.scale, in.plan) ||
      overlaps_any(st, sy, sb, sx, in.A, in.B, in.scale, in.plan) ||
      overlaps_any(sw, st, sy, sb, sx, in.A, in.B, in.scale, in.plan))
    return SQ_ERR_INVALID_ARG;
  LoraRequest q = {};
  SQ_TRY(device_word(&q.status));
  q.x = static_cast<const uint16_t *>(x);
  q.ldx = ldx;
  q.A = static_cast<const uint16_t *>(A);
  q.B = static_cast<const uint16_t *>(B);
  q.scale = scale;
  q.plan = plan;
  q.base = base;
  q.ld_base = base ? ldbase : 0;
  q.y = y;
  q.ldy = ldy;
  q.t = t;
  q.M = M;
  q.N = N;
  q.K = K;
  q.R = R;
  q.L = n_adapters;
  q.workspace = workspace;
  q.f32 = f32;
  return from_cuda(launch_lora_forward(q, cs(stream)));
}

sq_status sq_lora_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                           const float *t, const void *A, const void *B, const float *scale,
                           const int32_t *plan, const void *dx_base, int64_t ldbase, void *dx,
                           int64_t lddx, void *dA, void *dB, sq_out_dtype grad_dtype,
                           void *workspace, size_t workspace_bytes, int64_t M, int64_t N,
                           int64_t K, int32_t R, int32_t n_adapters, sq_stream_t stream) {
  if (grad_dtype != SQ_OUT_BF16 && grad_dtype != SQ_OUT_F32) return SQ_ERR_INVALID_ARG;
  SQ_TRY(check_lora(M, N, K, R, n_adapters, A, B, scale, plan));
  SQ_TRY(check_rows(dy, M, N, lddy));
  SQ_TRY(check_rows(x, M, K, ldx));
  if ((dA == nullptr) != (dB == nullptr)) return SQ_ERR_INVALID_ARG;
  if (dx == nullptr && dx_base != nullptr) return SQ_ERR_INVALID_ARG;
  if (dx != nullptr) SQ_TRY(check_rows(dx, M, K, lddx));
  if (dx_base != nullptr) SQ_TRY(check_rows(dx_base, M, K, ldbase));
  const bool f32 = grad_dtype == SQ_OUT_F32;
  if (M > 0 && (t == nullptr || workspace == nullptr ||
                workspace_bytes < lora_workspace_bytes(M, R, n_adapters, f32)))
    return SQ_ERR_INVALID_ARG;
  if (dx != nullptr && dx_base == dx && ldbase != lddx) return SQ_ERR_INVALID_ARG;
  if (dx != nullptr && M > 0 && (dx == dy || dx == x)) return SQ_ERR_INVALID_ARG;
  if (!aligned(t, 16) || !aligned(workspace, 16) || !aligned(dA, 16) || !aligned(dB, 16))
    return SQ_ERR_ALIGNMENT;
  if (dA == nullptr && (dx == nullptr || M == 0)) return SQ_OK;
  // The expansion reads A beside the outer products, which write dA and dB.
  const int64_t e = f32 ? 4 : 2, rank = static_cast<int64_t>(n_adapters) * R;
  const LoraSpans in(M, N, K, R, n_adapters, A, B, scale, plan);
  const Span sg(dy, M, N * 2, lddy * 2), sx(x, M, K * 2, ldx * 2), st(t, M * R * 4),
      sb(dx_base, dx_base ? M : 0, K * 2, ldbase * 2), sd(dx, dx ? M : 0, K * 2, lddx * 2),
      sA(dA, rank * K * e), sB(dB, rank * N * e),
      sw(workspace, lora_workspace_bytes(M, R, n_adapters, f32));
  if ((dx_base != dx && overlap(sd, sb)) ||
      overlaps_any(sd, sg, sx, st, in.A, in.B, in.scale, in.plan) || overlap(sA, sB) ||
      overlaps_any(sA, sd, sb, sg, sx, st, in.A, in.B, in.scale, in.plan) ||
      overlaps_any(sB, sd, sb, sg, sx, st, in.A, in.B, in.scale, in.plan) ||
      (M > 0 && overlaps_any(sw, sA, sB, sd, sb, sg, sx, st, in.A, in.B, in.scale, in.plan)))
    return SQ_ERR_INVALID_ARG;
  LoraRequest q = {};
  SQ_TRY(device_word(&q.status));
  q.x = static_cast<const uint16_t *>(x);
  q.ldx = ldx;
  q.dy = static_cast<const uint16_t *>(dy);
  q.lddy = lddy;
  q.A = static_cast<const uint16_t *>(A);
  q.B = static_cast<const uint16_t *>(B);
  q.scale = scale;
  q.plan = plan;
  q.base = dx_base;
  q.ld_base = dx_base ? ldbase : 0;
  q.dx = static_cast<uint16_t *>(dx);
  q.lddx = lddx;
  q.dA = dA;
  q.dB = dB;
  q.t = const_cast<float *>(t);
  q.workspace = workspace;
  q.M = M;
  q.N = N;
  q.K = K;
  q.R = R;
  q.L = n_adapters;
  q.f32 = f32;
  return from_cuda(launch_lora_backward(q, cs(stream)));
}

sq_status sq_rope_forward(const void *x, int64_t ldx, void *out, int64_t ldo, sq_out_dtype dtype,
                          const int32_t *positions, const float *inv_freq,
                          const int32_t *axis_pairs, int32_t n_axes, float factor, int64_t M,
                          int32_t H, int32_t D, int32_t rot, sq_rope_layout layout,
                          sq_stream_t stream) {
  return rope_common(x, ldx, out, ldo, dtype, positions, inv_freq, axis_pairs, n_axes, factor, M,
                     H, D, rot, layout, 1.0f, stream);
}

sq_status sq_rope_backward(const void *dout, int64_t lddo, void *dx, int64_t lddx,
                           sq_out_dtype dtype, const int32_t *positions, const float *inv_freq,
                           const int32_t *axis_pairs, int32_t n_axes, float factor, int64_t M,
                           int32_t H, int32_t D, int32_t rot, sq_rope_layout layout,
                           sq_stream_t stream) {
  return rope_common(dout, lddo, dx, lddx, dtype, positions, inv_freq, axis_pairs, n_axes, factor,
                     M, H, D, rot, layout, -1.0f, stream);
}

sq_status sq_rope_frequencies(int32_t rot, double base, sq_rope_scaling kind, double scale,
                              double original_context, double beta_fast, double beta_slow,
                              float *inv_freq, float *factor) {
  if (inv_freq == nullptr || factor == nullptr) return SQ_ERR_INVALID_ARG;
  if (rot < 2 || rot % 2 != 0 || rot > 1024) return SQ_ERR_INVALID_ARG;
  if (!(base > 1.0) || !isfinite(base) || !(scale >= 1.0) || !isfinite(scale))
    return SQ_ERR_INVALID_ARG;
  if (kind < SQ_ROPE_SCALE_NONE || kind > SQ_ROPE_SCALE_YARN) return SQ_ERR_INVALID_ARG;
  if (kind == SQ_ROPE_SCALE_NTK && rot <= 2) return SQ_ERR_INVALID_ARG;
  double lo = 0.0, hi = 0.0;
  if (kind == SQ_ROPE_SCALE_YARN) {
    if (!(original_context >= 1.0) || !isfinite(original_context) || !(beta_slow > 0.0) ||
        !(beta_fast > beta_slow) || !isfinite(beta_fast))
      return SQ_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    const double per = rot / (2.0 * log(base));
    lo = floor(per * log(original_context / (two_pi * beta_fast)));
    hi = ceil(per * log(original_context / (two_pi * beta_slow)));
    lo = fmin(fmax(lo, 0.0), rot - 1.0);
    hi = fmin(fmax(hi, 0.0), rot - 1.0);
    if (lo == hi) hi += 0.001;
  }
  if (kind == SQ_ROPE_SCALE_NTK) base *= pow(scale, rot / (rot - 2.0));
  *factor = kind == SQ_ROPE_SCALE_YARN && scale > 1.0 ? static_cast<float>(0.1 * log(scale) + 1.0)
                                                      : 1.0f;
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (kind == SQ_ROPE_SCALE_LINEAR) f /= scale;
    if (kind == SQ_ROPE_SCALE_YARN) {
      const double r = 1.0 - fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
      f *= (1.0 - r) / scale + r;
    }
    inv_freq[i] = static_cast<float>(f);
  }
  return SQ_OK;
}

size_t sq_group_norm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G) {
  return group_norm_sizes_ok(B, S, C, G) && B > 0 ? group_norm_workspace_bytes(B, S, C, G) : 0;
}

sq_status sq_group_norm_forward(const void *x, int64_t ldx, int64_t B, int64_t S, int64_t C,
                                int64_t G, const void *gamma, const void *beta, float eps,
                                sq_activation act, void *y, int64_t ldy, float *mean, float *rstd,
                                void *workspace, size_t workspace_bytes, sq_stream_t stream) {
  SQ_TRY(check_group_norm(B, S, C, G, gamma, beta, act, mean, rstd, workspace, workspace_bytes));
  if (!(eps >= 0.0f) || !isfinite(eps)) return SQ_ERR_INVALID_ARG;
  SQ_TRY(check_rows(x, B * S, C, ldx));
  SQ_TRY(check_rows(y, B * S, C, ldy));
  if (B == 0) return SQ_OK;
  if (x == y && ldx != ldy) return SQ_ERR_INVALID_ARG;
  const Span sx(x, B * S, C * 2, ldx * 2), sy(y, B * S, C * 2, ldy * 2), sg(gamma, C * 2),
      sb(beta, C * 2), sm(mean, B * G * 4), sr(rstd, B * G * 4),
      sw(workspace, group_norm_workspace_bytes(B, S, C, G));
  if ((x != y && overlap(sy, sx)) || overlaps_any(sy, sg, sb, sm, sr, sw) ||
      overlaps_any(sm, sr, sw, sx, sg, sb) || overlaps_any(sr, sw, sx, sg, sb) ||
      overlaps_any(sw, sx, sg, sb))
    return SQ_ERR_INVALID_ARG;
  int *status = nullptr;
  SQ_TRY(device_word(&status));
  GroupNormArgs p = group_norm_args(x, ldx, B, S, C, G, gamma, beta, mean, rstd, status);
  p.eps = eps;
  p.y = static_cast<uint16_t *>(y);
  p.ldy = ldy;
  return from_cuda(launch_group_norm_forward(p, workspace, act, cs(stream)));
}

sq_status sq_group_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                 int64_t B, int64_t S, int64_t C, int64_t G, const void *gamma,
                                 const void *beta, const float *mean, const float *rstd,
                                 sq_activation act, void *dx, int64_t lddx, void *dgamma,
                                 void *dbeta, sq_out_dtype grad_dtype, void *workspace,
                                 size_t workspace_bytes, sq_stream_t stream) {
  if (grad_dtype != SQ_OUT_BF16 && grad_dtype != SQ_OUT_F32) return SQ_ERR_INVALID_ARG;
  SQ_TRY(check_group_norm(B, S, C, G, gamma, beta, act, mean, rstd, workspace, workspace_bytes));
  SQ_TRY(check_rows(dy, B * S, C, lddy));
  SQ_TRY(check_rows(x, B * S, C, ldx));
  if (dx != nullptr) SQ_TRY(check_rows(dx, B * S, C, lddx));
  if (dx != nullptr && ((dx == dy && lddx != lddy) || dx == x)) return SQ_ERR_INVALID_ARG;
  const bool gf32 = grad_dtype == SQ_OUT_F32;
  if (!aligned(dgamma, gf32 ? 4 : 2) || !aligned(dbeta, gf32 ? 4 : 2)) return SQ_ERR_ALIGNMENT;
  if (dx == nullptr && dgamma == nullptr && dbeta == nullptr) return SQ_OK;
  const Span sd(dy, B * S, C * 2, lddy * 2), sx(x, B * S, C * 2, ldx * 2),
      so(dx, dx ? B * S : 0, C * 2, lddx * 2), sg(gamma, C * 2), sb(beta, C * 2),
      sm(mean, B * G * 4), sr(rstd, B * G * 4), sdg(dgamma, C * (gf32 ? 4 : 2)),
      sdb(dbeta, C * (gf32 ? 4 : 2)),
      sw(workspace, B > 0 ? group_norm_workspace_bytes(B, S, C, G) : 0);
  if ((dx != dy && overlap(so, sd)) || overlaps_any(so, sx, sg, sb, sm, sr) ||
      overlaps_any(sdg, sdb, so, sd, sx, sg, sb, sm, sr) ||
      overlaps_any(sdb, so, sd, sx, sg, sb, sm, sr) ||
      overlaps_any(sw, sdg, sdb, so, sd, sx, sg, sb, sm, sr))
    return SQ_ERR_INVALID_ARG;
  int *status = nullptr;
  SQ_TRY(device_word(&status));
  if (B == 0) {
    const size_t bytes = static_cast<size_t>(C) * (gf32 ? 4 : 2);
    for (void *g : {dgamma, dbeta})
      if (g != nullptr && cudaMemsetAsync(g, 0, bytes, cs(stream)) != cudaSuccess)
        return SQ_ERR_CUDA;
    return SQ_OK;
  }
  GroupNormArgs p = group_norm_args(x, ldx, B, S, C, G, gamma, beta, const_cast<float *>(mean),
                                    const_cast<float *>(rstd), status);
  p.dy = static_cast<const uint16_t *>(dy);
  p.lddy = lddy;
  p.dx = static_cast<uint16_t *>(dx);
  p.lddx = lddx;
  p.dgamma = dgamma;
  p.dbeta = dbeta;
  return from_cuda(launch_group_norm_backward(p, workspace, act, gf32, cs(stream)));
}

size_t sq_input_grad_workspace_bytes(int64_t N, int64_t K) {
  if (N < 1 || N > kMaxCols || K < 16 || K > kMaxCols || K % 16 != 0) return 0;
  return input_grad_workspace_bytes(N, K);
}

sq_status sq_dualscale_seglinear_input_grad(const void *dy, int64_t lddy, const int8_t *wq,
                                            const float *s_w, const float *d,
                                            const sq_segments *seg, void *dx, int64_t lddx,
                                            int64_t M, int64_t N, int64_t K, void *workspace,
                                            size_t workspace_bytes, sq_stream_t stream) {
  if (M < 0 || M > kMaxRows || N < 1 || N > kMaxCols || K < 16 || K > kMaxCols || K % 16 != 0)
    return SQ_ERR_INVALID_ARG;
  InputGradRequest r = {};
  SQ_TRY(parse_segments(seg, K, N, &r.seg));
  SQ_TRY(check_rows(dy, M, N, lddy));
  SQ_TRY(check_rows(dx, M, K, lddx));
  if (M == 0) return SQ_OK;
  if (wq == nullptr || s_w == nullptr || workspace == nullptr || dx == dy)
    return SQ_ERR_INVALID_ARG;
  if (workspace_bytes < input_grad_workspace_bytes(N, K)) return SQ_ERR_INVALID_ARG;
  if (!aligned(wq, 16) || !aligned(s_w, 4) || (d && !aligned(d, 4)) || !aligned(workspace, 256))
    return SQ_ERR_ALIGNMENT;
  const Span sg(dy, M, N * 2, lddy * 2), so(dx, M, K * 2, lddx * 2), swq(wq, N * K),
      ss(s_w, r.seg.S * N * 4), sd(d, d ? r.seg.G * K * 4 : 0),
      sw(workspace, input_grad_workspace_bytes(N, K));
  if (overlaps_any(so, sg, swq, ss, sd, sw) || overlaps_any(sw, sg, swq, ss, sd))
    return SQ_ERR_INVALID_ARG;
  SQ_TRY(device_word(&r.status));
  r.dy = static_cast<const uint16_t *>(dy);
  r.lddy = lddy;
  r.wq = wq;
  r.s_w = s_w;
  r.d = d;
  r.dx = static_cast<uint16_t *>(dx);
  r.lddx = lddx;
  r.workspace = workspace;
  r.M = M;
  r.N = N;
  r.K = K;
  return launch_input_grad(r, cs(stream));
}

}  // extern "C"
