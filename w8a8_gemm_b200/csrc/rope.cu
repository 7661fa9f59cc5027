// rope.cu -- rotary positions on the rows of a projection (the q|k columns of
// a QKV linear's output): of each head's D columns the first `rot` hold rot / 2
// pairs (u, v), and pair i of row m turns by the angle
//   phi = position[m][axis(i)] * inv_freq[i],
//   (u, v) -> factor (u cos phi - v sin phi, u sin phi + v cos phi);
// the backward pass turns by -phi.  Pairs are (x[2i], x[2i + 1]) or (x[i],
// x[i + rot / 2]).
//
// Bound by memory traffic: every element is read and written once.  A row's
// cosines and sines are the same for all of its heads, so a block computes
// them once into shared memory while its loads of the row are in flight.  The
// angle is formed and reduced to a fraction of a turn in fp64 (a position of a
// million times a frequency near one has an fp32 product that is off by 0.03
// rad); sine and cosine of the reduced angle are fp32.  9216 rows of 48 heads of
// 128, bf16: 38.2 us in a replayed graph on one input, 0.91 of the copy rate (51.7
// when a thread found its place in the row anew for every unit), 40.4 a call; 24
// rows of 32 heads: 2.5 us, 5.5 a call.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bf16.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows whose loads a thread has under way at once

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(w[j]);
      f[2 * j + 1] = bf16_hi(w[j]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]),
                      bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float load(const uint16_t *p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
  }
  static __device__ __forceinline__ void store(uint16_t *p, float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t *>(&b);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float load(const float *p) { return *p; }
  static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
};

// {cos, sin} of one pair, times the factor.
__device__ __forceinline__ float2 turn(const RopeArgs &p, int64_t row, int i) {
  int axis = 0;
  while (axis + 1 < p.axes && i >= p.axis_end[axis]) ++axis;
  const double turns = static_cast<double>(p.positions[row * p.axes + axis]) *
                       static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;
  const float f = static_cast<float>(turns - rint(turns));  // [-1/2, 1/2] of a turn
  float s, c;
  sincospif(2.0f * f, &s, &c);
  return make_float2(p.factor * c, p.sign * p.factor * s);
}

// HALF: 8-pair (fp32: 4-pair) units of two vectors, one from each half;
// interleaved: units of one vector of 4 (2) pairs.  The columns past `rot` are
// units of one vector that is copied (skipped when the rows are rotated in
// place).  VEC false: pairs and columns one by one, for rotated widths that
// are no multiple of a unit.
template <typename T, bool HALF, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
  extern __shared__ float2 cs[];  // [rows of the block][rot / 2]
  using V = Vec<T>;
  constexpr int N = V::N;
  const T *x = static_cast<const T *>(p.x);
  T *out = static_cast<T *>(p.out);
  const int pairs = p.rot / 2;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_block;
  const int rows = p.M - row0 < p.rows_per_block ? static_cast<int>(p.M - row0)
                                                 : p.rows_per_block;
  const bool in_place = p.x == p.out;

  auto angles = [&]() {
    for (int i = threadIdx.x; i < rows * pairs; i += kThreads)
      cs[i] = turn(p, row0 + i / pairs, i % pairs);
  };

  if constexpr (VEC) {
    // A thread keeps its place in the row (head, unit) over several rows; where
    // a row has fewer units than the block threads, `lanes` rows go side by side.
    const int turned = HALF ? pairs / N : p.rot / N;             // units of a head that turn
    const int per_head = turned + (in_place ? 0 : (p.D - p.rot) / N);
    const int per_row = p.H * per_head;
    const int lanes = per_row < kThreads ? kThreads / per_row : 1;
    const int lane = per_row < kThreads ? threadIdx.x / per_row : 0;
    int u = per_row < kThreads ? threadIdx.x - lane * per_row : threadIdx.x;
    int r = lane;
    bool work = lane < lanes && u < per_row && r < rows;
    int unit = 0;
    int64_t at = 0;  // element offset of the unit's first vector within a row
    uint4 a[kAhead], b[kAhead];
    auto place = [&]() {
      const int h = u / per_head;
      unit = u - h * per_head;
      at = static_cast<int64_t>(h) * p.D +
           (unit < turned ? unit * N : p.rot + (unit - turned) * N);
    };
    auto load = [&]() {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (r + q * lanes >= rows) break;
        const T *src = x + (row0 + r + q * lanes) * p.ldx + at;
        a[q] = *reinterpret_cast<const uint4 *>(src);
        if (HALF && unit < turned) b[q] = *reinterpret_cast<const uint4 *>(src + pairs);
      }
    };
    if (work) {
      place();
      load();
    }
    angles();
    __syncthreads();
    while (work) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (r + q * lanes >= rows) break;
        const int64_t row = row0 + r + q * lanes;
        T *dst = out + row * p.ldo + at;
        const int64_t end = at + (HALF && unit < turned ? pairs : 0) + N;  // columns
        const bool ok = store_ok(p.status, row < p.M && end <= static_cast<int64_t>(p.H) * p.D);
        if (unit >= turned) {
          if (ok) *reinterpret_cast<uint4 *>(dst) = a[q];
          continue;
        }
        const float4 *w = reinterpret_cast<const float4 *>(
            cs + (r + q * lanes) * pairs + unit * (HALF ? N : N / 2));  // two pairs each
        if constexpr (HALF) {
          float x0[N], x1[N], f0[N], f1[N];
          V::unpack(a[q], x0);
          V::unpack(b[q], x1);
#pragma unroll
          for (int j = 0; j < N; j += 2) {
            const float4 t = w[j / 2];
            f0[j] = x0[j] * t.x - x1[j] * t.y;
            f1[j] = x0[j] * t.y + x1[j] * t.x;
            f0[j + 1] = x0[j + 1] * t.z - x1[j + 1] * t.w;
            f1[j + 1] = x0[j + 1] * t.w + x1[j + 1] * t.z;
          }
          if (ok) {
            *reinterpret_cast<uint4 *>(dst) = V::pack(f0);
            *reinterpret_cast<uint4 *>(dst + pairs) = V::pack(f1);
          }
        } else {
          float x0[N], f[N];
          V::unpack(a[q], x0);
#pragma unroll
          for (int j = 0; j < N; j += 4) {
            const float4 t = w[j / 4];
            f[j] = x0[j] * t.x - x0[j + 1] * t.y;
            f[j + 1] = x0[j] * t.y + x0[j + 1] * t.x;
            f[j + 2] = x0[j + 2] * t.z - x0[j + 3] * t.w;
            f[j + 3] = x0[j + 2] * t.w + x0[j + 3] * t.z;
          }
          if (ok) *reinterpret_cast<uint4 *>(dst) = V::pack(f);
        }
      }
      r += kAhead * lanes;
      if (r >= rows) {
        r = lane;
        u += kThreads;
        work = per_row >= kThreads && u < per_row;
        if (work) place();
      }
      if (work) load();
    }
  } else {
    angles();
    __syncthreads();
    const int rest = in_place ? 0 : p.D - p.rot;
    const int per_head = pairs + rest;
    const int per_row = p.H * per_head;
    for (int u = threadIdx.x; u < rows * per_row; u += kThreads) {
      const int r = u / per_row, v = u - r * per_row;
      const int h = v / per_head, i = v - h * per_head;
      const T *src = x + (row0 + r) * p.ldx + static_cast<int64_t>(h) * p.D;
      T *dst = out + (row0 + r) * p.ldo + static_cast<int64_t>(h) * p.D;
      const int last = i >= pairs ? p.rot + i - pairs : HALF ? i + pairs : 2 * i + 1;
      if (!store_ok(p.status, row0 + r < p.M && last < p.D && h < p.H)) continue;
      if (i >= pairs) {
        dst[p.rot + i - pairs] = src[p.rot + i - pairs];
        continue;
      }
      const int iu = HALF ? i : 2 * i, iv = HALF ? i + pairs : 2 * i + 1;
      const float a = V::load(src + iu), b = V::load(src + iv);
      const float2 w = cs[r * pairs + i];
      V::store(dst + iu, a * w.x - b * w.y);
      V::store(dst + iv, a * w.y + b * w.x);
    }
  }
}

template <typename T>
cudaError_t run(RopeArgs p, bool half, cudaStream_t stream) {
  constexpr int N = Vec<T>::N;
  const bool vec = p.rot % (half ? 2 * N : N) == 0;
  // Rows of a block: enough for every thread to have an angle to form and its
  // loads under way, with at most 32 KB of cosines and sines, but no more than
  // leave every SM four blocks.
  const int64_t units = static_cast<int64_t>(p.H) * p.D / (vec && half ? 2 * N : N);
  int64_t rows = kThreads / (p.rot / 2);
  const int64_t ahead = units < kThreads ? kAhead * (kThreads / units) : kAhead;
  if (rows < ahead) rows = ahead;
  const int64_t most = 32768 / (static_cast<int64_t>(p.rot / 2) * 8);
  if (rows > most) rows = most;
  const int64_t blocks4 = 4 * static_cast<int64_t>(sm_count());
  if (rows > p.M / blocks4) rows = p.M / blocks4;
  if (rows < 1) rows = 1;
  p.rows_per_block = static_cast<int>(rows);
  const int64_t blocks = (p.M + rows - 1) / rows;
  const size_t smem = static_cast<size_t>(rows) * (p.rot / 2) * sizeof(float2);
  const unsigned g = static_cast<unsigned>(blocks);
  if (half && vec) rope_kernel<T, true, true><<<g, kThreads, smem, stream>>>(p);
  if (half && !vec) rope_kernel<T, true, false><<<g, kThreads, smem, stream>>>(p);
  if (!half && vec) rope_kernel<T, false, true><<<g, kThreads, smem, stream>>>(p);
  if (!half && !vec) rope_kernel<T, false, false><<<g, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &p, bool half, bool f32, cudaStream_t stream) {
  return f32 ? run<float>(p, half, stream) : run<uint16_t>(p, half, stream);
}

}  // namespace sq
