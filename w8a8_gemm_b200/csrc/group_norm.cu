// group_norm.cu -- group norm with an activation on channels-last rows, the
// producer of a quantized linear's input: x [B][S][C] (row stride ld), G groups
// of C / G neighbouring channels.
//   mean, var over the S x C/G values of a sample's group; rstd = 1/sqrt(var + eps)
//   v = (x - mean) rstd gamma + beta,  y = act(v)
// backward, with dv = dy act'(v), h = dv gamma, xh = (x - mean) rstd, n = S C/G:
//   dbeta = sum dv, dgamma = sum dv xh over samples and rows,
//   dx = rstd (h - (sum_group h + xh sum_group h xh) / n).
//
// Both directions take two kernels: one reads the rows and leaves partial results
// of its chunk of rows, the other joins the partials (a few KB) and reads the rows
// again, from L2 where they fit.  What bounds them is latency: two kernels one
// behind the other, at 16 to 24 warps an SM, which keep the issue slots and (two
// operations an element for SiLU and GELU) the special-function unit busy 35 to 45%
// of the time.  2 x 16384 x 320 with SiLU: 17.6 us in a replayed graph on one input,
// 20.2 a call with new ones; backward, 4 x 4096 x 640 with SiLU: 26.2 and 30.0.  (One
// kernel with the rows kept in a cluster's shared memory was measured: clusters
// of eight with 200 KB a block find room for 120 of 148 SMs, and the forward pass
// took 34 us in two rounds.)
//
// The statistics are (count, mean, sum of squares about the mean).  A thread sums
// x - c and (x - c)^2 over up to 32 rows, c the first of them, in fp32: the sum of
// squares is then off by at most 2^-23 n (c - mean)^2 for n = 32 rows, and since
// every c is one of the samples these add up to less than 2^-18 of the group's
// sum of squares, however far the mean lies above the deviation.  The joins are
// fp32, the last one fp64, all in a fixed order; they average the distances of the
// means from the first of them, so that a mean is off by its own roundings to
// fp32 and by the distances', and equal values have themselves for a mean.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bf16.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 8;     // rows whose loads a thread has under way in the statistics
constexpr int kShifted = 32;  // rows of one shifted sum: four batches
constexpr int kAhead = 4;     // and in the other kernels

__device__ __forceinline__ uint4 load8(const uint16_t *p) {
  return *reinterpret_cast<const uint4 *>(p);
}

// How a block's threads share C: `oct` octets of 8 channels a pass, `lanes`
// threads (rows) per octet.
struct Split {
  int oct, lanes;
};
__host__ __device__ inline Split split_of(int C) {
  const int o = C / 8;
  return o >= kThreads ? Split{kThreads, 1} : Split{o, kThreads / o};
}

// f(q) for the first `n` of K rows: without a test for each where there are K, so
// that the rows' instructions mix.
template <int K, typename F>
__device__ __forceinline__ void first_rows(int n, F &&f) {
  if (n >= K) {
#pragma unroll
    for (int q = 0; q < K; ++q) f(q);
  } else {
#pragma unroll
    for (int q = 0; q < K - 1; ++q)
      if (q < n) f(q);
  }
}
// f(e, group of channel c0 + e) for eight channels, with one division.
template <typename F>
__device__ __forceinline__ void eight_groups(int c0, int cg, F &&f) {
  int g = c0 / cg, left = (g + 1) * cg - c0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f(e, g);
    if (--left == 0) {
      left = cg;
      ++g;
    }
  }
}
// Rows lane, lane + lanes, ... below `rows`.
__device__ __forceinline__ int rows_of(int lane, int lanes, int rows) {
  return lane < lanes && lane < rows ? (rows - 1 - lane) / lanes + 1 : 0;
}

// 2^u and 1/u by the special-function unit, within 2^-22 or so; past the largest
// number inf and 0.  (The library's quick exponential and division take care of
// denormal numbers too, at four times the instructions.)
__device__ __forceinline__ float exp2_quick(float u) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(u));
  return r;
}
__device__ __forceinline__ float rcp_quick(float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(u));
  return r;
}
__device__ __forceinline__ F2 splat(float v) { return f2(v, v); }

// SiLU is v sigmoid(u) with u = v, tanh GELU with u = 2 sqrt(2/pi) (v + 0.044715
// v^3); sigmoid(u) = 1 / (1 + 2^(-u log2 e)).
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGelu = 1.5957691216057308f, kGelu3 = kGelu * 0.044715f;  // 2 sqrt(2/pi)
template <int ACT>
__device__ __forceinline__ F2 gate(F2 v) {
  F2 u;
  if constexpr (ACT == SQ_ACT_GELU)
    u = f2_mul(v, f2_fma(f2_mul(v, v), splat(-kGelu3 * kLog2E), splat(-kGelu * kLog2E)));
  else
    u = f2_mul(v, splat(-kLog2E));
  const float2 w = f2_get(u);
  const float2 d = f2_get(f2_add(f2(exp2_quick(w.x), exp2_quick(w.y)), splat(1.0f)));
  return f2(rcp_quick(d.x), rcp_quick(d.y));
}
template <int ACT>
__device__ __forceinline__ F2 act(F2 v) {
  if constexpr (ACT == SQ_ACT_NONE) return v;
  return f2_mul(v, gate<ACT>(v));
}
// (v g(u))' = g (1 + v u' (1 - g)).  GELU: g (1 - g) v first, which is 0 where |v| is
// large, whose cube (v u') may be past the largest number.
template <int ACT>
__device__ __forceinline__ F2 act_grad(F2 v) {
  const F2 g = gate<ACT>(v), rest = f2_fma(g, splat(-1.0f), splat(1.0f));
  if constexpr (ACT == SQ_ACT_GELU)
    return f2_fma(f2_mul(f2_mul(g, rest), v),
                  f2_fma(f2_mul(v, v), splat(3.0f * kGelu3), splat(kGelu)), g);
  return f2_mul(g, f2_fma(v, rest, splat(1.0f)));
}

// Running statistics of eight channels over the rows a thread has seen.
struct Running {
  F2 mean[4], m2[4];
  float n;
  __device__ __forceinline__ void clear() {
    n = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) mean[j] = m2[j] = f2(0.0f, 0.0f);
  }
  // joins `rows` rows of mean bm and squares bs about it
  __device__ __forceinline__ void join(float rows, const F2 (&bm)[4], const F2 (&bs)[4]) {
    // the quick quotient need not be 1 where there was nothing to join
    const float total = n + rows, w = n > 0.0f ? __fdividef(rows, total) : 1.0f;
    const F2 w2 = f2(w, w), nw = f2(n * w, n * w), minus = f2(-1.0f, -1.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const F2 delta = f2_fma(mean[j], minus, bm[j]);
      mean[j] = f2_fma(delta, w2, mean[j]);
      m2[j] = f2_fma(f2_mul(delta, delta), nw, f2_add(m2[j], bs[j]));
    }
    n = total;
  }
  // {mean, squares} of each channel
  __device__ __forceinline__ void store(float2 *to) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = f2_get(mean[j]), b = f2_get(m2[j]);
      reinterpret_cast<float4 *>(to)[j] = make_float4(a.x, b.x, a.y, b.y);
    }
  }
};

// Sums over the channels of each group of f(c), a power of two of neighbouring
// threads per group: out(g, sum) by one of them, or all with ALL.
__host__ __device__ inline int threads_per_group(int cg) {
  int t = 1;
  while (t < 32 && t * 8 < cg) t *= 2;
  return t;
}
__device__ __forceinline__ float2 sum_over(float2 s, int t) {
  for (int o = 1; o < t; o <<= 1) {
    s.x += __shfl_xor_sync(~0u, s.x, o);
    s.y += __shfl_xor_sync(~0u, s.y, o);
  }
  return s;
}

// Joins the threads' statistics sh[lanes][width] (lane l saw the rows l, l + lanes,
// ... of `rows`), {mean, squares} of each channel, over the lanes into chan[width]
// and these over each group into out(g, mean, squares): first the mean, then the
// squares about it.
template <typename Out>
__device__ __forceinline__ void join_lanes(const float2 *sh, float2 *chan, int lanes, int width,
                                           int rows, int groups, int cg, Out &&out) {
  const int each = rows / lanes, more = rows % lanes;  // rows of a lane
  const int used = rows < lanes ? rows : lanes;        // lanes with any
  const float all = static_cast<float>(rows), inv = 1.0f / all;
  __syncthreads();
  for (int c = threadIdx.x; c < width; c += kThreads) {
    const float pivot = sh[c].x;
    float s = 0.0f;
    for (int l = 1; l < used; ++l)
      s = fmaf(static_cast<float>(each + (l < more)), sh[l * width + c].x - pivot, s);
    const float mean = fmaf(s, inv, pivot);
    float m2 = 0.0f;
    for (int l = 0; l < used; ++l) {
      const float2 v = sh[l * width + c];
      const float d = v.x - mean;
      m2 += fmaf(static_cast<float>(each + (l < more)) * d, d, v.y);
    }
    chan[c] = make_float2(mean, m2);
  }
  __syncthreads();
  const int t = threads_per_group(cg), part = threadIdx.x % t;
  for (int g0 = 0; g0 < groups; g0 += kThreads / t) {
    const int g = g0 + threadIdx.x / t;
    const float2 *src = chan + g * cg;
    float2 s = make_float2(0.0f, 0.0f);
    const float pivot = g < groups ? src[0].x : 0.0f;
    if (g < groups)
      for (int c = part; c < cg; c += t) s.x += src[c].x - pivot;
    const float mean = pivot + sum_over(s, t).x / static_cast<float>(cg);
    s.x = 0.0f;
    if (g < groups)
      for (int c = part; c < cg; c += t) {
        const float2 v = src[c];
        const float d = v.x - mean;
        s.y += fmaf(all * d, d, v.y);
      }
    const float m2 = sum_over(s, t).y;
    if (g < groups && part == 0) out(g, mean, m2);
  }
}

// chan[c] = sum over l of sh[l][c], c < width, by all threads in a fixed order.
template <int THREADS>
__device__ __forceinline__ void channel_sums(float2 *sh, float2 *chan, int lanes, int width) {
  __syncthreads();
  if (width > THREADS) {  // few lanes
    for (int c = threadIdx.x; c < width; c += THREADS) {
      float2 s = sh[c];
      for (int l = 1; l < lanes; ++l) {
        s.x += sh[l * width + c].x;
        s.y += sh[l * width + c].y;
      }
      chan[c] = s;
    }
  } else {
    const int parts = THREADS / width < lanes ? THREADS / width : lanes;
    const int part = threadIdx.x / width, c = threadIdx.x % width;
    float2 s = make_float2(0.0f, 0.0f);
    if (part < parts)
      for (int l = part; l < lanes; l += parts) {
        s.x += sh[l * width + c].x;
        s.y += sh[l * width + c].y;
      }
    __syncthreads();
    if (part < parts) sh[part * width + c] = s;
    __syncthreads();
    if (part == 0) {
      for (int q = 1; q < parts; ++q) {
        s.x += sh[q * width + c].x;
        s.y += sh[q * width + c].y;
      }
      chan[c] = s;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------- forward
// Chunk statistics: part[b][chunk][g] = {mean, sum of squares about it}.
__global__ void __launch_bounds__(kThreads, 2) gn_stats_kernel(const GroupNormArgs p) {
  // [lanes][C] {mean, squares} of each thread's rows, then of all rows
  extern __shared__ float2 sh[];
  grid_dependency_wait();
  grid_dependency_launch();
  const int b = blockIdx.y;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_chunk;
  const int rows = p.S - r0 < p.rows_per_chunk ? static_cast<int>(p.S - r0) : p.rows_per_chunk;
  const Split sp = split_of(p.C);
  const int lane = threadIdx.x / sp.oct, oct = threadIdx.x % sp.oct;
  const uint16_t *x = p.x + (static_cast<int64_t>(b) * p.S + r0) * p.ldx;
  for (int o = oct; o < p.C / 8 && lane < sp.lanes; o += sp.oct) {
    Running st;
    st.clear();
    const int64_t step = sp.lanes * p.ldx;
    const uint16_t *src = x + lane * p.ldx + o * 8;
    uint4 v[kBatch];
    auto load = [&](int n) {
      first_rows<kBatch>(n, [&](int q) { v[q] = load8(src + q * step); });
      src += kBatch * step;
    };
    int left = rows_of(lane, sp.lanes, rows);
    load(left);
    while (left > 0) {
      // sums of x - c and (x - c)^2 over up to kShifted rows, c the first of them
      const F2 minus = splat(-1.0f);
      const F2 c[4] = {f2_mul(f2_of_bf16(v[0].x), minus), f2_mul(f2_of_bf16(v[0].y), minus),
                       f2_mul(f2_of_bf16(v[0].z), minus), f2_mul(f2_of_bf16(v[0].w), minus)};
      F2 s[4], s2[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = s2[j] = splat(0.0f);
      const int n = left < kShifted ? left : kShifted;
      for (int i = 0; i < n; i += kBatch, left -= kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) w[q] = v[q];
        load(left - kBatch);
        first_rows<kBatch>(left, [&](int q) {
          const uint32_t u[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const F2 d = f2_add(f2_of_bf16(u[j]), c[j]);
            s[j] = f2_add(s[j], d);
            s2[j] = f2_fma(d, d, s2[j]);
          }
        });
      }
      const float inv = __fdividef(1.0f, static_cast<float>(n));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 m = f2_mul(s[j], splat(inv));
        s2[j] = f2_fma(f2_mul(s[j], minus), m, s2[j]);
        s[j] = f2_fma(c[j], minus, m);
      }
      st.join(static_cast<float>(n), s, s2);
    }
    st.store(sh + lane * p.C + o * 8);
  }
  const int64_t slot = (static_cast<int64_t>(b) * p.chunks + blockIdx.x) * p.G;
  join_lanes(sh, sh + sp.lanes * p.C, sp.lanes, p.C, rows, p.G, p.C / p.G,
             [&](int g, float mean, float m2) {
               if (store_ok(p.status, slot + g < static_cast<int64_t>(p.B) * p.chunks * p.G))
                 p.part[slot + g] = make_float2(mean, m2);
             });
}

// Sums over a sample's chunks of {f(v, n), g(v, n)} of each group's partials, n
// rows in the chunk, in fp64: all threads load (thread t: group t % G of every
// (t / G)-th chunk), and a group's partial sums are added in a fixed order.
// `sums` [kThreads] in shared memory; ends with sums[g] ready for all.
template <typename F>
__device__ __forceinline__ void chunk_sums(const GroupNormArgs &p, int b, double2 *sums, int g0,
                                           int width, F &&f) {
  const int lanes = kThreads / width;
  const int g = threadIdx.x % width, l = threadIdx.x / width;
  double2 s = make_double2(0.0, 0.0);
  if (l < lanes) {
    const float2 *src = p.part + static_cast<int64_t>(b) * p.chunks * p.G + g0 + g;
#pragma unroll 4
    for (int k = l; k < p.chunks; k += lanes) {
      const float2 v = src[static_cast<int64_t>(k) * p.G];
      const double2 a = f(v, k + 1 < p.chunks ? p.rows_per_chunk
                                              : p.S - static_cast<int64_t>(k) * p.rows_per_chunk);
      s.x += a.x;
      s.y += a.y;
    }
  }
  __syncthreads();  // the last user of `sums` is done
  if (l < lanes) sums[l * width + g] = s;
  __syncthreads();
  if (threadIdx.x < width) {
    for (int q = 1; q < lanes; ++q) {
      s.x += sums[q * width + g].x;
      s.y += sums[q * width + g].y;
    }
    sums[g] = s;
  }
  __syncthreads();
}

// Joins a sample's chunk statistics into {mean, rstd} of `groups` groups.  Means are
// taken from the first chunk's: the squares about it are at most (1 + q) times the
// variance, q = (distance of the first chunk's mean / deviation)^2 at most the number
// of chunks (a chunk is a share of the rows), so that fp64 loses 2^-40 of it.
__device__ __forceinline__ void join_stats(const GroupNormArgs &p, int b, int first, int groups,
                                           float2 *stat, double2 *sums) {
  const double cg = p.C / p.G, n = static_cast<double>(p.S);
  for (int g0 = 0; g0 < groups; g0 += kThreads) {
    const int width = groups - g0 < kThreads ? groups - g0 : kThreads;
    const double pivot =
        p.part[static_cast<int64_t>(b) * p.chunks * p.G + first + g0 + threadIdx.x % width].x;
    chunk_sums(p, b, sums, first + g0, width, [&](float2 v, double rows) {
      const double m = v.x - pivot;
      return make_double2(rows * m, v.y + rows * cg * m * m);
    });
    if (threadIdx.x < width) {
      const double m = sums[threadIdx.x].x / n;
      double var = sums[threadIdx.x].y / (n * cg) - m * m;
      if (var < 0.0) var = 0.0;
      stat[g0 + threadIdx.x] =
          make_float2(static_cast<float>(pivot + m),
                      static_cast<float>(1.0 / sqrt(var + static_cast<double>(p.eps))));
    }
  }
  __syncthreads();
}

// A thread's first rows are under way before the statistics are there: x was
// complete before the statistics' kernel began to read it.  Four rows a thread and
// the channels' values in registers fit three blocks an SM without spills (eight
// rows: 2 x 16384 x 320 in 18.7 us, four: 17.6).
template <int ACT>
__global__ void __launch_bounds__(kThreads, 3) gn_apply_kernel(const GroupNormArgs p) {
  extern __shared__ float2 sh[];  // {mean, rstd} of the slice's groups
  __shared__ double2 sums[kThreads];
  const int b = blockIdx.y, cg = p.C / p.G;
  const int ch0 = blockIdx.z * p.slice;
  const int width = p.C - ch0 < p.slice ? p.C - ch0 : p.slice;
  const int first = ch0 / cg, groups = width / cg;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows2;
  const int rows = p.S - r0 < p.rows2 ? static_cast<int>(p.S - r0) : p.rows2;
  const Split sp = split_of(width);
  const int lane = threadIdx.x / sp.oct, oct = threadIdx.x % sp.oct;
  const int64_t row0 = static_cast<int64_t>(b) * p.S + r0;
  const int mine = rows_of(lane, sp.lanes, rows);
  const int64_t stepx = sp.lanes * p.ldx, stepy = sp.lanes * p.ldy;
  const uint16_t *x = p.x + (row0 + lane) * p.ldx;
  uint4 v[kAhead];
  auto load = [&](const uint16_t *src, int n) {
    first_rows<kAhead>(n, [&](int q) { v[q] = load8(src + q * stepx); });
  };
  // the channels' gamma and beta, as they lie in two bf16 of a word
  uint32_t gm[4], bt[4];
  auto load_params = [&](int c0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + 2 * j;
      gm[j] = p.gamma ? p.gamma[c] | static_cast<uint32_t>(p.gamma[c + 1]) << 16 : 0x3F803F80u;
      bt[j] = p.beta ? p.beta[c] | static_cast<uint32_t>(p.beta[c + 1]) << 16 : 0u;
    }
  };
  bool loaded = lane < sp.lanes;
  if (loaded) {
    load(x + ch0 + oct * 8, mine);
    load_params(ch0 + oct * 8);
  }
  grid_dependency_wait();
  join_stats(p, b, first, groups, sh, sums);
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g < groups; g += kThreads)
      if (store_ok(p.status, b * p.G + first + g < p.B * p.G)) {
        p.mean[b * p.G + first + g] = sh[g].x;
        p.rstd[b * p.G + first + g] = sh[g].y;
      }
  if (lane >= sp.lanes) return;
  for (int o = oct; o < width / 8; o += sp.oct) {
    const int c0 = ch0 + o * 8;
    if (o != oct) load_params(c0);
    // (x - mean) scale + beta, as the backward pass has it: x scale + (beta - mean
    // scale) would cancel where the mean is far above the deviation
    F2 scale[4], minus_mean[4], beta[4];
    float k[8], m[8];
    eight_groups(c0, cg, [&](int e, int g) {
      const float2 st = sh[g - first];
      k[e] = st.y * (e & 1 ? bf16_hi(gm[e / 2]) : bf16_lo(gm[e / 2]));
      m[e] = -st.x;
    });
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      scale[j] = f2(k[2 * j], k[2 * j + 1]);
      minus_mean[j] = f2(m[2 * j], m[2 * j + 1]);
      beta[j] = f2_of_bf16(bt[j]);
    }
    const uint16_t *src = x + c0;
    uint16_t *dst = p.y + (row0 + lane) * p.ldy + c0;
    const uint16_t *end = p.y + (static_cast<int64_t>(p.B) * p.S - 1) * p.ldy + p.C;
    for (int left = mine; left > 0; left -= kAhead) {
      if (!loaded) load(src, left);
      loaded = false;
      first_rows<kAhead>(left, [&](int q) {
        const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 d = f2_add(f2_of_bf16(w[j]), minus_mean[j]);
          const float2 z = f2_get(act<ACT>(f2_fma(d, scale[j], beta[j])));
          y[j] = bf16x2(z.x, z.y);
        }
        if (store_ok(p.status, c0 + 8 <= p.C && dst + q * stepy + 8 <= end))
          *reinterpret_cast<uint4 *>(dst + q * stepy) = make_uint4(y[0], y[1], y[2], y[3]);
      });
      src += kAhead * stepx;
      dst += kAhead * stepy;
    }
  }
}

// ------------------------------------------------------------------ backward
// The fixed values of a thread's eight channels.
struct Octet {
  F2 minus_mean[4], rstd[4], gamma[4], beta[4];
  __device__ __forceinline__ void load(const GroupNormArgs &p, int b, int c0, int cg) {
    float m[8], r[8], gm[8], bt[8];
    eight_groups(c0, cg, [&](int e, int g) {
      m[e] = -p.mean[b * p.G + g];
      r[e] = p.rstd[b * p.G + g];
      gm[e] = p.gamma ? bf16_lo(p.gamma[c0 + e]) : 1.0f;
      bt[e] = p.beta ? bf16_lo(p.beta[c0 + e]) : 0.0f;
    });
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      minus_mean[j] = f2(m[2 * j], m[2 * j + 1]);
      rstd[j] = f2(r[2 * j], r[2 * j + 1]);
      gamma[j] = f2(gm[2 * j], gm[2 * j + 1]);
      beta[j] = f2(bt[2 * j], bt[2 * j + 1]);
    }
  }
  // xh and dv of the channels 2 j, 2 j + 1
  template <int ACT>
  __device__ __forceinline__ void at(uint32_t x, uint32_t dy, int j, F2 &xh, F2 &dv) const {
    xh = f2_mul(f2_add(f2_of_bf16(x), minus_mean[j]), rstd[j]);
    dv = f2_of_bf16(dy);
    if constexpr (ACT != SQ_ACT_NONE)
      dv = f2_mul(dv, act_grad<ACT>(f2_fma(xh, gamma[j], beta[j])));
  }
};

template <bool GF32>
__device__ __forceinline__ void store_param_grads(const GroupNormArgs &p, int c, float s, float sx) {
  if (!store_ok(p.status, c >= 0 && c < p.C)) return;
  if constexpr (GF32) {
    if (p.dgamma) static_cast<float *>(p.dgamma)[c] = sx;
    if (p.dbeta) static_cast<float *>(p.dbeta)[c] = s;
  } else {
    if (p.dgamma) static_cast<__nv_bfloat16 *>(p.dgamma)[c] = __float2bfloat16_rn(sx);
    if (p.dbeta) static_cast<__nv_bfloat16 *>(p.dbeta)[c] = __float2bfloat16_rn(s);
  }
}

// Chunk sums: chan_part[b][chunk][c] = {sum dv, sum dv xh} and
// part[b][chunk][g] = {sum h, sum h xh}.
template <int ACT>
__global__ void __launch_bounds__(kThreads, 2) gn_bwd_sums_kernel(const GroupNormArgs p) {
  extern __shared__ float2 sh[];  // [lanes][C], then the channels' sums
  grid_dependency_wait();
  grid_dependency_launch();
  const int b = blockIdx.y;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_chunk;
  const int rows = p.S - r0 < p.rows_per_chunk ? static_cast<int>(p.S - r0) : p.rows_per_chunk;
  const Split sp = split_of(p.C);
  const int lane = threadIdx.x / sp.oct, oct = threadIdx.x % sp.oct;
  const int cg = p.C / p.G;
  const int64_t row0 = static_cast<int64_t>(b) * p.S + r0;
  const int64_t slot = static_cast<int64_t>(b) * p.chunks + blockIdx.x;

  for (int o = oct; o < p.C / 8 && lane < sp.lanes; o += sp.oct) {
    const int c0 = o * 8;
    Octet ch;
    ch.load(p, b, c0, cg);
    F2 sd[4], sx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sd[j] = sx[j] = f2(0.0f, 0.0f);
    const int64_t stepx = sp.lanes * p.ldx, stepd = sp.lanes * p.lddy;
    const uint16_t *xs = p.x + (row0 + lane) * p.ldx + c0;
    const uint16_t *ds = p.dy + (row0 + lane) * p.lddy + c0;
    for (int left = rows_of(lane, sp.lanes, rows); left > 0; left -= kAhead) {
      uint4 vx[kAhead], vd[kAhead];
      first_rows<kAhead>(left, [&](int q) {
        vx[q] = load8(xs + q * stepx);
        vd[q] = load8(ds + q * stepd);
      });
      xs += kAhead * stepx;
      ds += kAhead * stepd;
      first_rows<kAhead>(left, [&](int q) {
        const uint32_t x[4] = {vx[q].x, vx[q].y, vx[q].z, vx[q].w};
        const uint32_t d[4] = {vd[q].x, vd[q].y, vd[q].z, vd[q].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          F2 xh, dv;
          ch.at<ACT>(x[j], d[j], j, xh, dv);
          sd[j] = f2_add(sd[j], dv);
          sx[j] = f2_fma(dv, xh, sx[j]);
        }
      });
    }
    float4 *to = reinterpret_cast<float4 *>(sh + lane * p.C + c0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = f2_get(sd[j]), v = f2_get(sx[j]);
      to[j] = make_float4(u.x, v.x, u.y, v.y);
    }
  }
  float2 *chan = sh + sp.lanes * p.C;
  channel_sums<kThreads>(sh, chan, sp.lanes, p.C);
  for (int c = threadIdx.x; c < p.C; c += kThreads)
    if (store_ok(p.status, slot * p.C + c < static_cast<int64_t>(p.B) * p.chunks * p.C))
      p.chan_part[slot * p.C + c] = chan[c];
  const int n = threads_per_group(cg), part = threadIdx.x % n;
  for (int g0 = 0; g0 < p.G; g0 += kThreads / n) {
    const int g = g0 + threadIdx.x / n;
    float2 s = make_float2(0.0f, 0.0f);
    if (g < p.G)
      for (int c = g * cg + part; c < (g + 1) * cg; c += n) {
        const float gm = p.gamma ? bf16_lo(p.gamma[c]) : 1.0f;
        s.x = fmaf(gm, chan[c].x, s.x);
        s.y = fmaf(gm, chan[c].y, s.y);
      }
    s = sum_over(s, n);
    if (g < p.G && part == 0 &&
        store_ok(p.status, slot * p.G + g < static_cast<int64_t>(p.B) * p.chunks * p.G))
      p.part[slot * p.G + g] = s;
  }
}

// The first `grad_blocks` blocks add up 32 channels each of dgamma and dbeta;
// the others write dx.
template <int ACT, bool GF32>
__global__ void __launch_bounds__(kThreads, 2) gn_bwd_dx_kernel(const GroupNormArgs p) {
  extern __shared__ float2 sh[];
  __shared__ double2 sums[kThreads];
  const int warp = threadIdx.x >> 5, ln = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < p.grad_blocks) {
    grid_dependency_wait();
    const int c = blockIdx.x * 32 + ln;
    double s = 0.0, sx = 0.0;
    if (c < p.C) {
#pragma unroll 8
      for (int64_t k = warp; k < static_cast<int64_t>(p.B) * p.chunks; k += kWarps) {
        const float2 v = p.chan_part[k * p.C + c];
        s += v.x;
        sx += v.y;
      }
    }
    sums[warp * 32 + ln] = make_double2(s, sx);
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < kWarps; ++w) {
      s += sums[w * 32 + ln].x;
      sx += sums[w * 32 + ln].y;
    }
    if (c < p.C) store_param_grads<GF32>(p, c, static_cast<float>(s), static_cast<float>(sx));
    return;
  }
  const int blk = blockIdx.x - p.grad_blocks;
  const int chunk = blk % p.chunks2, b = blk / p.chunks2 % p.B;
  const int cg = p.C / p.G;
  const int ch0 = blk / p.chunks2 / p.B * p.slice;
  const int width = p.C - ch0 < p.slice ? p.C - ch0 : p.slice;
  const int first = ch0 / cg, groups = width / cg;
  const int64_t r0 = static_cast<int64_t>(chunk) * p.rows2;
  const int rows = p.S - r0 < p.rows2 ? static_cast<int>(p.S - r0) : p.rows2;
  const Split sp = split_of(width);
  const int lane = threadIdx.x / sp.oct, oct = threadIdx.x % sp.oct;
  const int64_t row0 = static_cast<int64_t>(b) * p.S + r0;
  // The first rows and values of the channels come before the sums: they were
  // complete before the sums' kernel began to read them.
  uint4 vx[kAhead], vd[kAhead];
  Octet ch;
  const int mine = rows_of(lane, sp.lanes, rows);
  const int64_t stepx = sp.lanes * p.ldx, stepd = sp.lanes * p.lddy, stepo = sp.lanes * p.lddx;
  auto load = [&](const uint16_t *xs, const uint16_t *ds, int n) {
    first_rows<kAhead>(n, [&](int q) {
      vx[q] = load8(xs + q * stepx);
      vd[q] = load8(ds + q * stepd);
    });
  };
  const uint16_t *x0 = p.x + (row0 + lane) * p.ldx + ch0;
  const uint16_t *d0 = p.dy + (row0 + lane) * p.lddy + ch0;
  bool loaded = lane < sp.lanes;
  if (loaded) {
    load(x0 + oct * 8, d0 + oct * 8, mine);
    ch.load(p, b, ch0 + oct * 8, cg);
  }
  grid_dependency_wait();
  const double n = static_cast<double>(p.S) * cg;
  // group sums over -n
  for (int g0 = 0; g0 < groups; g0 += kThreads) {
    const int n_now = groups - g0 < kThreads ? groups - g0 : kThreads;
    chunk_sums(p, b, sums, first + g0, n_now,
               [](float2 v, double) { return make_double2(v.x, v.y); });
    if (threadIdx.x < n_now)
      sh[g0 + threadIdx.x] = make_float2(static_cast<float>(-sums[threadIdx.x].x / n),
                                         static_cast<float>(-sums[threadIdx.x].y / n));
  }
  __syncthreads();
  if (lane >= sp.lanes) return;
  for (int o = oct; o < width / 8; o += sp.oct) {
    const int c0 = ch0 + o * 8;
    if (o != oct) ch.load(p, b, c0, cg);
    F2 m1[4], m2[4];
    float s1[8], s2[8];
    eight_groups(c0, cg, [&](int e, int g) {
      s1[e] = sh[g - first].x;
      s2[e] = sh[g - first].y;
    });
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m1[j] = f2(s1[2 * j], s1[2 * j + 1]);
      m2[j] = f2(s2[2 * j], s2[2 * j + 1]);
    }
    const uint16_t *xs = x0 + o * 8, *ds = d0 + o * 8;
    uint16_t *dst = p.dx + (row0 + lane) * p.lddx + c0;
    const uint16_t *end = p.dx + (static_cast<int64_t>(p.B) * p.S - 1) * p.lddx + p.C;
    for (int left = mine; left > 0; left -= kAhead) {
      if (!loaded) load(xs, ds, left);
      loaded = false;
      first_rows<kAhead>(left, [&](int q) {
        const uint32_t x[4] = {vx[q].x, vx[q].y, vx[q].z, vx[q].w};
        const uint32_t d[4] = {vd[q].x, vd[q].y, vd[q].z, vd[q].w};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          F2 xh, dv;
          ch.at<ACT>(x[j], d[j], j, xh, dv);
          const float2 z =
              f2_get(f2_mul(ch.rstd[j], f2_fma(xh, m2[j], f2_fma(dv, ch.gamma[j], m1[j]))));
          y[j] = bf16x2(z.x, z.y);
        }
        if (store_ok(p.status, c0 + 8 <= p.C && dst + q * stepo + 8 <= end))
          *reinterpret_cast<uint4 *>(dst + q * stepo) = make_uint4(y[0], y[1], y[2], y[3]);
      });
      xs += kAhead * stepx;
      ds += kAhead * stepd;
      dst += kAhead * stepo;
    }
  }
}

// ------------------------------------------------------------------ host side
// Rows of a chunk: two blocks per SM of a 148-SM device over all samples, but at
// least four rows per thread where S allows.  Fewer, longer chunks also mean
// fewer partials to join in every block of the second kernel.  A fixed rule, so
// that the workspace size and the order of every sum depend on the sizes only.
int64_t chunk_rows(int64_t B, int64_t S, int64_t C) {
  const int64_t want = (2 * 148 + B - 1) / B;
  const int64_t lanes = split_of(static_cast<int>(C)).lanes;
  const int64_t rows = (S + want - 1) / want;
  return rows > 4 * lanes ? rows : 4 * lanes;
}

// Shared memory of the first kernels: every thread's eight channels (or all
// channels, where they are more), and two floats per channel.
int lane_smem(int C) { return (split_of(C).lanes + 1) * C * static_cast<int>(sizeof(float2)); }

// Launch behind the kernel ahead in the stream (programmatic dependent launch:
// every kernel here waits for it before it reads anything).
template <auto Kernel>
cudaError_t launch(dim3 grid, size_t smem, size_t max_smem, const GroupNormArgs &p,
                   cudaStream_t stream) {
  static bool done[64] = {};  // per kernel and device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(max_smem));
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, Kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr size_t kMaxLaneSmem = kGroupNormMaxC * 2 * sizeof(float2);
constexpr size_t kMaxGroupSmem = kGroupNormMaxG * sizeof(float2);

void fill_chunks(GroupNormArgs &p, int blocks2) {
  p.rows_per_chunk = static_cast<int32_t>(chunk_rows(p.B, p.S, p.C));
  p.chunks = static_cast<int32_t>((p.S + p.rows_per_chunk - 1) / p.rows_per_chunk);
  // A block of the second kernel has a slice of the channels, whole octets and
  // whole groups, eight groups or 128 bytes a row at least: every block joins its
  // groups' partials of the whole sample before it starts (all 32 groups of
  // 2 x 16384 x 320 in every block: 23.1 us, eight: 19.0 us then).
  const int cg = p.C / p.G;
  const int unit = cg % 8 == 0 ? cg : cg % 4 == 0 ? cg * 2 : cg % 2 == 0 ? cg * 4 : cg * 8;
  const int least_width = 8 * cg > 64 ? 8 * cg : 64;
  const int width = (least_width + unit - 1) / unit * unit;
  p.slice = width < p.C ? width : p.C;
  p.slices = (p.C + p.slice - 1) / p.slice;
  // Its rows: the blocks that an SM holds at once (three forward, two backward) in
  // one round beside the blocks of dgamma and dbeta, but at least four rows per
  // thread.
  const int64_t each = static_cast<int64_t>(p.B) * p.slices;
  int64_t want = (blocks2 * 148 - p.grad_blocks) / each;
  if (want < 1) want = 1;
  const int64_t least = 4 * split_of(p.slice).lanes;
  const int64_t rows = (p.S + want - 1) / want;
  p.rows2 = static_cast<int32_t>(rows > least ? rows : least);
  p.chunks2 = static_cast<int32_t>((p.S + p.rows2 - 1) / p.rows2);
}

template <int ACT>
cudaError_t run_forward(const GroupNormArgs &p, cudaStream_t stream) {
  const cudaError_t e =
      launch<gn_stats_kernel>(dim3(p.chunks, p.B), lane_smem(p.C), kMaxLaneSmem, p, stream);
  if (e != cudaSuccess) return e;
  return launch<gn_apply_kernel<ACT>>(dim3(p.chunks2, p.B, p.slices),
                                      p.slice / (p.C / p.G) * sizeof(float2), kMaxGroupSmem, p,
                                      stream);
}

template <int ACT>
cudaError_t run_backward(GroupNormArgs p, bool gf32, cudaStream_t stream) {
  const cudaError_t e = launch<gn_bwd_sums_kernel<ACT>>(dim3(p.chunks, p.B), lane_smem(p.C),
                                                        kMaxLaneSmem, p, stream);
  if (e != cudaSuccess) return e;
  const int grid = p.grad_blocks + (p.dx ? p.chunks2 * p.B * p.slices : 0);
  if (grid == 0) return cudaSuccess;
  const size_t smem = p.G * sizeof(float2);
  return gf32 ? launch<gn_bwd_dx_kernel<ACT, true>>(dim3(grid), smem, kMaxGroupSmem, p, stream)
              : launch<gn_bwd_dx_kernel<ACT, false>>(dim3(grid), smem, kMaxGroupSmem, p, stream);
}

}  // namespace

// float2 words: group partials, then (backward) channel partials.
size_t group_norm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G) {
  const int64_t rows = chunk_rows(B, S, C);
  const int64_t chunks = (S + rows - 1) / rows;
  return static_cast<size_t>(B * chunks * (G + C)) * sizeof(float2);
}

cudaError_t launch_group_norm_forward(GroupNormArgs p, void *workspace, int act,
                                      cudaStream_t stream) {
  fill_chunks(p, 3);
  p.part = static_cast<float2 *>(workspace);
  if (act == SQ_ACT_SILU) return run_forward<SQ_ACT_SILU>(p, stream);
  if (act == SQ_ACT_GELU) return run_forward<SQ_ACT_GELU>(p, stream);
  return run_forward<SQ_ACT_NONE>(p, stream);
}

cudaError_t launch_group_norm_backward(GroupNormArgs p, void *workspace, int act, bool gf32,
                                       cudaStream_t stream) {
  p.grad_blocks = (p.dgamma || p.dbeta) ? (p.C + 31) / 32 : 0;
  fill_chunks(p, 2);
  p.part = static_cast<float2 *>(workspace);
  p.chan_part = p.part + static_cast<int64_t>(p.B) * p.chunks * p.G;
  if (act == SQ_ACT_SILU) return run_backward<SQ_ACT_SILU>(p, gf32, stream);
  if (act == SQ_ACT_GELU) return run_backward<SQ_ACT_GELU>(p, gf32, stream);
  return run_backward<SQ_ACT_NONE>(p, gf32, stream);
}

}  // namespace sq
