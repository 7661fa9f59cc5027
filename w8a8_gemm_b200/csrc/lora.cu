// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   t[m] = A[a] x[m]                 (rank R)        y[m] = base[m] + c[a] B[a] t[m]
//   dt[m] = c[a] B[a]^T dy[m]                        dx[m] = dx_base[m] + A[a]^T dt[m]
//   dB[a] = c[a] sum_{m of a} dy[m] t[m]^T           dA[a] = sum_{m of a} dt[m] x[m]^T
//
// with a = adapter[m].  A plan, made once per batch, lists the rows adapter by
// adapter and cuts them into tiles of at most 64 rows of one adapter, so that
// every tile is an ordinary pair of thin matrix products whatever the order of
// the rows: scattered rows are gathered, single tokens of one adapter share a
// tile, and the plan serves every layer that the batch goes through.
//
// Three kernels:
//   contract  [rows] x [C] -> [rows] x R: t (rows of A) and dt (columns of B);
//   expand    [rows] x R -> [rows] x [C] added to base: y and dx;
//   outer     [rows] x [C], [rows] x R -> [C] x R: dB and dA.
// All are bound by the rows' traffic (at rank 64 a row element that is read
// and written, four bytes, meets 128 flop); the products run on the warp-level
// matrix path, whose rate suffices up to rank 128.  Sums are fp32; the small
// operand t (dt) is kept in fp32 and enters the second product as bf16 where
// the result is rounded to bf16 anyway, or split into three bf16 terms (24
// significant bits) where the result stays fp32.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mma.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

namespace cg = cooperative_groups;

constexpr int kTileRows = SQ_LORA_TILE_ROWS;
constexpr int32_t kPlanMagic = 0x53514C31;
constexpr int kThreads = 256;

// ------------------------------------------------------------------- the plan
// int32 words: [0] magic, [1] M, [2] L, [3] tiles, then bin_start[L + 2] (bin L
// holds the rows without an adapter), perm[M] (rows, adapter by adapter, in
// ascending order within one), tiles[max_tiles] of {bin, first place in perm}.
struct PlanView {
  const int32_t *head, *bin_start, *perm, *tiles;
};
__host__ __device__ inline int64_t plan_perm_at(int32_t L) { return 4 + (L + 2); }
__host__ __device__ inline int64_t plan_tiles_at(int64_t M, int32_t L) {
  return plan_perm_at(L) + M;
}
__host__ __device__ inline int64_t plan_max_tiles(int64_t M, int32_t L) {
  return M / kTileRows + (M < L + 1 ? M : L + 1);
}
__device__ __forceinline__ PlanView plan_view(const int32_t *plan, int64_t M, int32_t L) {
  return {plan, plan + 4, plan + plan_perm_at(L), plan + plan_tiles_at(M, L)};
}
// A plan of another batch size or adapter count: reported, nothing computed.
__device__ __forceinline__ bool plan_fits(const PlanView &v, int64_t M, int32_t L, int *status) {
  const bool ok = v.head[0] == kPlanMagic && v.head[1] == static_cast<int32_t>(M) &&
                  v.head[2] == L;
  if (!ok && threadIdx.x == 0) atomicCAS(status, 0, static_cast<int>(SQ_ERR_INVALID_ARG));
  return ok;
}

// One block: a stable counting sort of the rows by adapter.  Warp w owns the
// rows [w chunk, (w + 1) chunk) and a histogram of its own, so that the order
// within an adapter, and with it every sum over its rows, is always the same.
constexpr int kPlanWarps = 32;
__global__ void __launch_bounds__(kPlanWarps * 32) lora_plan_kernel(
    const int32_t *__restrict__ adapter, int32_t M, int32_t L, int32_t *plan, int *status) {
  extern __shared__ int32_t sh[];
  const int bins = L + 1;
  int32_t *hist = sh;                        // [kPlanWarps][bins]
  int32_t *start = sh + kPlanWarps * bins;   // [bins + 1] rows before a bin
  int32_t *tile_at = start + bins + 1;       // [bins + 1] tiles before a bin
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * bins; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  const int chunk = ((M + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
  const int64_t lo = static_cast<int64_t>(warp) * chunk;
  const int64_t hi = lo + chunk < M ? lo + chunk : M;
  int32_t *mine = hist + warp * bins;
  for (int64_t r = lo + lane; r < hi; r += 32) {
    const int32_t a = adapter[r];
    atomicAdd(&mine[a >= 0 && a < L ? a : L], 1);
  }
  __syncthreads();
  // rows of each bin, and each warp's first place within it
  for (int b = threadIdx.x; b < bins; b += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int n = hist[w * bins + b];
      hist[w * bins + b] = sum;
      sum += n;
    }
    start[b] = sum;
  }
  __syncthreads();
  // exclusive prefix over the bins (one warp, 32 bins a step)
  if (warp == 0) {
    int rows = 0, tiles = 0;
    for (int b0 = 0; b0 < bins; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < bins ? start[b] : 0;
      const int nt = (n + kTileRows - 1) / kTileRows;
      int sr = n, st = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int ur = __shfl_up_sync(~0u, sr, o), ut = __shfl_up_sync(~0u, st, o);
        if (lane >= o) {
          sr += ur;
          st += ut;
        }
      }
      if (b < bins) {
        start[b] = rows + sr - n;
        tile_at[b] = tiles + st - nt;
      }
      rows += __shfl_sync(~0u, sr, 31);
      tiles += __shfl_sync(~0u, st, 31);
    }
    if (lane == 0) {
      start[bins] = rows;
      tile_at[bins] = tiles;
    }
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    const int32_t v[4] = {kPlanMagic, M, L, tile_at[bins]};
    if (store_ok(status, threadIdx.x < plan_perm_at(L))) plan[threadIdx.x] = v[threadIdx.x];
  }
  for (int b = threadIdx.x; b <= bins; b += blockDim.x)
    if (store_ok(status, 4 + b < plan_perm_at(L))) plan[4 + b] = start[b];
  int32_t *tiles = plan + plan_tiles_at(M, L);
  const int64_t max_tiles = plan_max_tiles(M, L);
  for (int b = warp; b < bins; b += kPlanWarps)
    for (int i = lane; i < tile_at[b + 1] - tile_at[b]; i += 32) {
      const int64_t at = tile_at[b] + i;
      if (!store_ok(status, at < max_tiles)) continue;
      tiles[2 * at] = b;
      tiles[2 * at + 1] = start[b] + i * kTileRows;
    }
  // places: 32 rows a step in order; equal bins of a step rank by lane
  int32_t *perm = plan + plan_perm_at(L);
  for (int64_t r0 = lo; r0 < hi; r0 += 32) {
    const int64_t r = r0 + lane;
    const bool in = r < hi;
    const int32_t a = in ? adapter[r] : 0;
    const int b = !in ? -1 : (a >= 0 && a < L ? a : L);
    const unsigned same = __match_any_sync(~0u, b);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (in) {
      const int64_t at = start[b] + mine[b] + rank;
      if (store_ok(status, at >= 0 && at < M)) perm[at] = static_cast<int32_t>(r);
    }
    __syncwarp();
    if (in && rank == 0) mine[b] += __popc(same);
    __syncwarp();
  }
}

// ----------------------------------------------------------------- shared parts
// A tile's rows: bin, first place, count; false past the last tile.
struct Tile {
  int bin, start, count;
};
__device__ __forceinline__ bool get_tile(const PlanView &v, int i, Tile &t) {
  if (i >= v.head[3]) return false;
  t.bin = v.tiles[2 * i];
  t.start = v.tiles[2 * i + 1];
  const int left = v.bin_start[t.bin + 1] - t.start;
  t.count = left < kTileRows ? left : kTileRows;
  return true;
}

// Byte offset of 16-byte chunk c of row r in a tile of 128-byte rows, chunks
// exchanged within groups of eight rows so that ldmatrix meets no bank twice.
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// ------------------------------------------------------------------- contract
// out[m][j] = f sum_c in[m][c] W(j, c), f = scale[a] or 1; W(j, c) = w[a][j][c]
// (TRANS false: A) or w[a][c][j] (TRANS true: B).  One block per row tile and
// slice of the contracted dimension; the blocks of a cluster hold the slices
// of one tile and add their partial sums through distributed shared memory in
// a fixed order.
struct ContractArgs {
  const uint16_t *in;
  int64_t ld;
  const uint16_t *w;
  const float *scale;  // nullptr: 1
  const int32_t *plan;
  float *out;
  int64_t M;
  int32_t C, R, L;
  int *status;
};

template <int RT, bool TRANS>
struct ContractSmem {
  static constexpr int kStages = 4;
  static constexpr int kIn = kTileRows * 128;
  static constexpr int kWRow = TRANS ? RT * 2 + 16 : 128;
  static constexpr int kW = TRANS ? 64 * kWRow : RT * 128;
  static constexpr int kStage = kIn + kW;
  static constexpr int kRows = kStages * kStage;  // then the tile's row numbers
  static constexpr int kBytes = kRows + kTileRows * 4;
  static_assert(kTileRows * (RT + 1) * 4 <= kRows, "partial sums reuse the stages");
};

template <int RT, bool TRANS>
__global__ void __launch_bounds__(kThreads) lora_contract_kernel(const ContractArgs p) {
  using S = ContractSmem<RT, TRANS>;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int slices = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const PlanView plan = plan_view(p.plan, p.M, p.L);
  if (!plan_fits(plan, p.M, p.L, p.status)) return;
  Tile t;
  if (!get_tile(plan, blockIdx.x, t) || t.bin >= p.L) return;  // the whole cluster returns

  int32_t *rows = reinterpret_cast<int32_t *>(smem + S::kRows);
  for (int i = threadIdx.x; i < kTileRows; i += kThreads)
    rows[i] = plan.perm[t.start + (i < t.count ? i : 0)];
  __syncthreads();

  const int C = p.C;
  const int slice = ((C + slices - 1) / slices + 63) / 64 * 64;
  const int c_lo = rank * slice;
  const int c_hi = c_lo + slice < C ? c_lo + slice : C;
  const int steps = c_hi > c_lo ? (c_hi - c_lo + 63) / 64 : 0;
  const uint16_t *w = p.w + static_cast<int64_t>(t.bin) * p.R * C;
  const uint32_t base = smem_u32(smem);

  auto load = [&](int step) {
    const uint32_t st = base + (step % S::kStages) * S::kStage;
    const int c0 = c_lo + step * 64;
    for (int i = threadIdx.x; i < kTileRows * 8; i += kThreads) {
      const int r = i >> 3, c = i & 7;
      const int col = c0 + c * 8;
      const bool ok = r < t.count && col < c_hi;
      cp_async16(st + swz(r, c), p.in + rows[r] * p.ld + (ok ? col : 0), ok);
    }
    const uint32_t sw = st + S::kIn;
    if constexpr (!TRANS) {
      for (int i = threadIdx.x; i < RT * 8; i += kThreads) {
        const int r = i >> 3, c = i & 7;
        const int col = c0 + c * 8;
        const bool ok = r < p.R && col < c_hi;
        cp_async16(sw + swz(r, c), ok ? w + static_cast<int64_t>(r) * C + col : w, ok);
      }
    } else {
      for (int i = threadIdx.x; i < 64 * (RT / 8); i += kThreads) {
        const int r = i / (RT / 8), c = i % (RT / 8);
        const int row = c0 + r;
        const bool ok = row < c_hi && c * 8 < p.R;
        cp_async16(sw + r * S::kWRow + c * 16,
                   ok ? w + static_cast<int64_t>(row) * p.R + c * 8 : w, ok);
      }
    }
  };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp & 3, wn = warp >> 2;
  constexpr int NT = RT / 16;  // n tiles of 8 columns per warp (half of RT)
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;

#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (s < steps) load(s);
    cp_async_commit();
  }
  for (int step = 0; step < steps; ++step) {
    cp_async_wait<S::kStages - 2>();
    __syncthreads();
    if (step + S::kStages - 1 < steps) load(step + S::kStages - 1);
    cp_async_commit();
    if (wm * 16 >= t.count) continue;  // no rows in this warp's part
    const uint32_t si = base + (step % S::kStages) * S::kStage;
    const uint32_t sw = si + S::kIn;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t a[4];
      ldsm_x4(si + swz(wm * 16 + (lane & 15), kk * 2 + (lane >> 4)), a);
      if constexpr (NT == 1) {
        uint32_t b0, b1;
        if constexpr (!TRANS)
          ldsm_x2(sw + swz(wn * 8 + (lane & 7), kk * 2 + ((lane >> 3) & 1)), b0, b1);
        else
          ldsm_x2_t(sw + (kk * 16 + (lane & 15)) * S::kWRow + wn * 16, b0, b1);
        mma_bf16(acc[0], a, b0, b1);
      } else {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          const int col = wn * (RT / 2) + n * 8;
          if constexpr (!TRANS)
            ldsm_x4(sw + swz(col + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)),
                    b);
          else
            ldsm_x4_t(sw + (kk * 16 + (lane & 15)) * S::kWRow + (col + (lane >> 4) * 8) * 2, b);
          mma_bf16(acc[n], a, b[0], b[1]);
          mma_bf16(acc[n + 1], a, b[2], b[3]);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // partial sums -> shared memory [64][RT + 1] -> sum over the slices
  float *part = reinterpret_cast<float *>(smem);
  constexpr int PS = RT + 1;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = wn * (RT / 2) + n * 8 + (lane & 3) * 2;
    const int row = wm * 16 + (lane >> 2);
    part[row * PS + col] = acc[n][0];
    part[row * PS + col + 1] = acc[n][1];
    part[(row + 8) * PS + col] = acc[n][2];
    part[(row + 8) * PS + col + 1] = acc[n][3];
  }
  if (slices > 1) cluster.sync(); else __syncthreads();
  const float f = p.scale ? p.scale[t.bin] : 1.0f;
  const int total = t.count * p.R;
  for (int e = rank * kThreads + threadIdx.x; e < total; e += slices * kThreads) {
    const int r = e / p.R, j = e - r * p.R;
    float s = 0.0f;
    for (int q = 0; q < slices; ++q) {
      const float *src = slices > 1 ? cluster.map_shared_rank(part, q) : part;
      s += src[r * PS + j];
    }
    const int64_t at = static_cast<int64_t>(rows[r]) * p.R + j;
    if (store_ok(p.status, rows[r] >= 0 && rows[r] < p.M && j < p.R)) p.out[at] = f * s;
  }
  if (slices > 1) cluster.sync();  // no block leaves while its sums are read
}

// --------------------------------------------------------------------- expand
// out[m][c] = base[m][c] + f sum_j t[m][j] W(j, c); W(j, c) = w[a][c][j] (TRANS
// false: B) or w[a][j][c] (TRANS true: A).  One block per row tile and 128
// output columns.  Rows without an adapter are copied from base (left alone
// when out is base).
struct ExpandArgs {
  const float *t;
  const uint16_t *w;
  const float *scale;  // nullptr: 1
  const int32_t *plan;
  const void *base;    // nullptr: 0
  int64_t ld_base;
  void *out;
  int64_t ld_out;
  int64_t M;
  int32_t C, R, L;
  int *status;
};

constexpr int kSlab = 128;

template <int RT, bool TRANS, bool F32>
struct ExpandSmem {
  static constexpr int kTerms = F32 ? 3 : 1;  // bf16 terms of t
  static constexpr int kTRow = RT * 2 + 16;
  static constexpr int kT = kTerms * kTileRows * kTRow;
  static constexpr int kWRow = TRANS ? kSlab * 2 + 16 : RT * 2 + 16;
  static constexpr int kW = TRANS ? RT * kWRow : kSlab * kWRow;
  static constexpr int kElem = F32 ? 4 : 2;
  static constexpr int kORow = kSlab * kElem + 16;
  static constexpr int kOut = kTileRows * kORow;
  static constexpr int kRows = kT + kW + kOut;
  static constexpr int kBytes = kRows + kTileRows * 4;
};

template <int RT, bool TRANS, bool F32>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(const ExpandArgs p) {
  using S = ExpandSmem<RT, TRANS, F32>;
  extern __shared__ __align__(128) uint8_t smem[];
  const PlanView plan = plan_view(p.plan, p.M, p.L);
  if (!plan_fits(plan, p.M, p.L, p.status)) return;
  const unsigned slabs = (static_cast<unsigned>(p.C) + kSlab - 1) / kSlab;
  Tile t;
  if (!get_tile(plan, static_cast<int>(blockIdx.x / slabs), t)) return;
  const bool none = t.bin >= p.L;
  if (none && p.base == p.out) return;

  constexpr int E = S::kElem;
  constexpr int VE = 16 / E;            // elements of a 16-byte chunk
  constexpr int CH = kSlab / VE;        // chunks of a row
  uint8_t *st = smem, *sw = smem + S::kT, *so = smem + S::kT + S::kW;
  int32_t *rows = reinterpret_cast<int32_t *>(smem + S::kRows);
  for (int i = threadIdx.x; i < kTileRows; i += kThreads)
    rows[i] = plan.perm[t.start + (i < t.count ? i : 0)];
  __syncthreads();
  const int c0 = static_cast<int>(blockIdx.x % slabs) * kSlab;

  // base tile and weight slab, asynchronously
  for (int i = threadIdx.x; i < kTileRows * CH; i += kThreads) {
    const int r = i / CH, c = i % CH;
    const bool ok = p.base != nullptr && r < t.count && c0 + c * VE < p.C;
    const uint8_t *src = static_cast<const uint8_t *>(p.base) +
                         (rows[r] * p.ld_base + (ok ? c0 + c * VE : 0)) * E;
    cp_async16(smem_u32(so + r * S::kORow + c * 16), ok ? src : static_cast<const void *>(p.t), ok);
  }
  if (!none) {
    const uint16_t *w = p.w + static_cast<int64_t>(t.bin) * p.R * p.C;
    if constexpr (!TRANS) {
      for (int i = threadIdx.x; i < kSlab * (RT / 8); i += kThreads) {
        const int r = i / (RT / 8), c = i % (RT / 8);
        const bool ok = c0 + r < p.C && c * 8 < p.R;
        cp_async16(smem_u32(sw + r * S::kWRow + c * 16),
                   ok ? w + static_cast<int64_t>(c0 + r) * p.R + c * 8 : w, ok);
      }
    } else {
      for (int i = threadIdx.x; i < RT * (kSlab / 8); i += kThreads) {
        const int r = i / (kSlab / 8), c = i % (kSlab / 8);
        const bool ok = r < p.R && c0 + c * 8 < p.C;
        cp_async16(smem_u32(sw + r * S::kWRow + c * 16),
                   ok ? w + static_cast<int64_t>(r) * p.C + c0 + c * 8 : w, ok);
      }
    }
    // t rows -> bf16 terms
    for (int i = threadIdx.x; i < kTileRows * (RT / 4); i += kThreads) {
      const int r = i / (RT / 4), c = i % (RT / 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r < t.count && c * 4 < p.R)
        v = *reinterpret_cast<const float4 *>(p.t + static_cast<int64_t>(rows[r]) * p.R + c * 4);
#pragma unroll
      for (int s = 0; s < S::kTerms; ++s) {
        const uint32_t lo = bf16x2(v.x, v.y), hi = bf16x2(v.z, v.w);
        *reinterpret_cast<uint2 *>(st + s * kTileRows * S::kTRow + r * S::kTRow + c * 8) =
            make_uint2(lo, hi);
        v = make_float4(v.x - bf16_lo(lo), v.y - bf16_hi(lo), v.z - bf16_lo(hi),
                        v.w - bf16_hi(hi));
      }
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncthreads();

  if (!none) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wm = warp & 3, wn = warp >> 2;
    if (wm * 16 < t.count) {
      float acc[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll
      for (int s = S::kTerms - 1; s >= 0; --s) {  // the smallest terms first
#pragma unroll
        for (int kk = 0; kk < RT / 16; ++kk) {
          uint32_t a[4];
          ldsm_x4(smem_u32(st + s * kTileRows * S::kTRow + (wm * 16 + (lane & 15)) * S::kTRow +
                           (kk * 16 + (lane >> 4) * 8) * 2),
                  a);
#pragma unroll
          for (int n = 0; n < 8; n += 2) {
            uint32_t b[4];
            const int col = wn * 64 + n * 8;
            if constexpr (!TRANS)
              ldsm_x4(smem_u32(sw + (col + (lane & 7) + ((lane >> 4) << 3)) * S::kWRow +
                               (kk * 16 + ((lane >> 3) & 1) * 8) * 2),
                      b);
            else
              ldsm_x4_t(smem_u32(sw + (kk * 16 + (lane & 15)) * S::kWRow +
                                 (col + (lane >> 4) * 8) * 2),
                        b);
            mma_bf16(acc[n], a, b[0], b[1]);
            mma_bf16(acc[n + 1], a, b[2], b[3]);
          }
        }
      }
      const float f = p.scale ? p.scale[t.bin] : 1.0f;
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = wm * 16 + (lane >> 2) + h * 8;
          const int col = wn * 64 + n * 8 + (lane & 3) * 2;
          uint8_t *at = so + row * S::kORow + col * E;
          const float u = acc[n][2 * h], v = acc[n][2 * h + 1];
          if constexpr (F32) {
            float2 o = *reinterpret_cast<float2 *>(at);
            o.x = fmaf(f, u, o.x);
            o.y = fmaf(f, v, o.y);
            *reinterpret_cast<float2 *>(at) = o;
          } else {
            const uint32_t o = *reinterpret_cast<uint32_t *>(at);
            *reinterpret_cast<uint32_t *>(at) =
                bf16x2(fmaf(f, u, bf16_lo(o)), fmaf(f, v, bf16_hi(o)));
          }
        }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < t.count * CH; i += kThreads) {
    const int r = i / CH, c = i % CH;
    if (c0 + c * VE >= p.C) continue;
    uint8_t *dst =
        static_cast<uint8_t *>(p.out) + (rows[r] * p.ld_out + c0 + c * VE) * E;
    if (store_ok(p.status, rows[r] >= 0 && rows[r] < p.M && c0 + c * VE + VE <= p.ld_out))
      *reinterpret_cast<uint4 *>(dst) =
          *reinterpret_cast<const uint4 *>(so + r * S::kORow + c * 16);
  }
}

// ---------------------------------------------------------------------- outer
// out[a](c, j) = f sum_{m of a} src[m][c] v[m][j]: dB[a][n][j] (src dy, v t, f =
// scale) and dA[a][j][k] (src x, v dt, f = 1, stored transposed).  One block
// per adapter, 64 columns c and share of the adapter's row tiles; the blocks
// of a cluster hold the shares and add them in a fixed order.
struct OuterSide {
  const uint16_t *src;
  int64_t ld;
  const float *v;
  const float *scale;  // nullptr: 1
  void *out;
  int32_t C;
  int32_t transposed;  // out [R][C] instead of [C][R]
};
struct OuterArgs {
  OuterSide side[2];
  int32_t slabs0;  // slabs of side 0
  const int32_t *plan;
  int64_t M;
  int32_t R, L;
  int *status;
};

template <int RT, bool F32>
struct OuterSmem {
  static constexpr int kTerms = F32 ? 3 : 1;
  static constexpr int kStages = 4;
  static constexpr int kSrc = kTileRows * 128;
  static constexpr int kVRow = RT * 2 + 16;
  static constexpr int kV = kTerms * kTileRows * kVRow;  // two buffers
  static constexpr int kVAt = kStages * kSrc;
  static constexpr int kPart = 64 * (RT + 1) * 4;
  static constexpr int kBuf = kVAt + 2 * kV;
  static constexpr int kBytes = kBuf > kPart ? kBuf : kPart;
};

template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads) lora_outer_kernel(const OuterArgs p) {
  using S = OuterSmem<RT, F32>;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int shares = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const PlanView plan = plan_view(p.plan, p.M, p.L);
  if (!plan_fits(plan, p.M, p.L, p.status)) return;
  const int bin = blockIdx.y;
  const bool second = static_cast<int>(blockIdx.x) >= p.slabs0;
  const OuterSide &sd = p.side[second ? 1 : 0];
  const int c0 = (static_cast<int>(blockIdx.x) - (second ? p.slabs0 : 0)) * 64;
  const int first = plan.bin_start[bin], end = plan.bin_start[bin + 1];
  const int tiles = (end - first + kTileRows - 1) / kTileRows;
  const int steps = tiles > rank ? (tiles - rank + shares - 1) / shares : 0;
  const uint32_t base = smem_u32(smem);

  auto load = [&](int step) {
    const int at = first + (rank + step * shares) * kTileRows;
    const uint32_t st = base + (step % S::kStages) * S::kSrc;
    for (int i = threadIdx.x; i < kTileRows * 8; i += kThreads) {
      const int r = i >> 3, c = i & 7;
      const bool ok = at + r < end && c0 + c * 8 < sd.C;
      const int64_t row = ok ? plan.perm[at + r] : 0;
      cp_async16(st + swz(r, c), sd.src + (ok ? row * sd.ld + c0 + c * 8 : 0), ok);
    }
  };
  // this thread's part of a tile of v: RT / 16 groups of four values
  constexpr int VN = kTileRows * (RT / 4) / kThreads;
  float4 vr[VN];
  auto fetch_v = [&](int step) {
    const int at = first + (rank + step * shares) * kTileRows;
#pragma unroll
    for (int q = 0; q < VN; ++q) {
      const int i = threadIdx.x + q * kThreads;
      const int r = i / (RT / 4), c = i % (RT / 4);
      vr[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (at + r < end && c * 4 < p.R)
        vr[q] = *reinterpret_cast<const float4 *>(
            sd.v + static_cast<int64_t>(plan.perm[at + r]) * p.R + c * 4);
    }
  };
  auto store_v = [&](int buf) {
#pragma unroll
    for (int q = 0; q < VN; ++q) {
      const int i = threadIdx.x + q * kThreads;
      const int r = i / (RT / 4), c = i % (RT / 4);
      float4 v = vr[q];
#pragma unroll
      for (int s = 0; s < S::kTerms; ++s) {
        const uint32_t lo = bf16x2(v.x, v.y), hi = bf16x2(v.z, v.w);
        *reinterpret_cast<uint2 *>(smem + S::kVAt + buf * S::kV +
                                   (s * kTileRows + r) * S::kVRow + c * 8) = make_uint2(lo, hi);
        v = make_float4(v.x - bf16_lo(lo), v.y - bf16_hi(lo), v.z - bf16_lo(hi),
                        v.w - bf16_hi(hi));
      }
    }
  };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp & 3, wn = warp >> 2;
  constexpr int NT = RT / 16;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;

#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (s < steps) load(s);
    cp_async_commit();
  }
  if (steps > 0) fetch_v(0);
  for (int step = 0; step < steps; ++step) {
    store_v(step & 1);  // the buffer read two steps ago
    cp_async_wait<S::kStages - 2>();
    __syncthreads();
    if (step + S::kStages - 1 < steps) load(step + S::kStages - 1);
    cp_async_commit();
    if (step + 1 < steps) fetch_v(step + 1);
    const uint32_t ss = base + (step % S::kStages) * S::kSrc;
    const uint32_t sv = base + S::kVAt + (step & 1) * S::kV;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      // source columns are the product's rows: transposed fragments
      uint32_t a[4];
      ldsm_x4_t(ss + swz(kk * 16 + (lane & 7) + ((lane >> 4) << 3), wm * 2 + ((lane >> 3) & 1)),
                a);
#pragma unroll
      for (int s = S::kTerms - 1; s >= 0; --s) {
        const uint32_t vrow = sv + (s * kTileRows + kk * 16 + (lane & 15)) * S::kVRow;
        if constexpr (NT == 1) {
          uint32_t b0, b1;
          ldsm_x2_t(vrow + wn * 16, b0, b1);
          mma_bf16(acc[0], a, b0, b1);
        } else {
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm_x4_t(vrow + (wn * (RT / 2) + n * 8 + (lane >> 4) * 8) * 2, b);
            mma_bf16(acc[n], a, b[0], b[1]);
            mma_bf16(acc[n + 1], a, b[2], b[3]);
          }
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  float *part = reinterpret_cast<float *>(smem);
  constexpr int PS = RT + 1;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = wn * (RT / 2) + n * 8 + (lane & 3) * 2;
    const int row = wm * 16 + (lane >> 2);
    part[row * PS + col] = acc[n][0];
    part[row * PS + col + 1] = acc[n][1];
    part[(row + 8) * PS + col] = acc[n][2];
    part[(row + 8) * PS + col + 1] = acc[n][3];
  }
  if (shares > 1) cluster.sync(); else __syncthreads();
  const float f = sd.scale ? sd.scale[bin] : 1.0f;
  const int cols = sd.C - c0 < 64 ? sd.C - c0 : 64;
  const int total = cols * p.R;
  const int64_t obase = static_cast<int64_t>(bin) * p.R * sd.C;
  for (int e = rank * kThreads + threadIdx.x; e < total; e += shares * kThreads) {
    int c, j;
    if (sd.transposed) {
      j = e / cols;
      c = e - j * cols;
    } else {
      c = e / p.R;
      j = e - c * p.R;
    }
    float s = 0.0f;
    for (int q = 0; q < shares; ++q) {
      const float *src = shares > 1 ? cluster.map_shared_rank(part, q) : part;
      s += src[c * PS + j];
    }
    const int64_t at = obase + (sd.transposed ? static_cast<int64_t>(j) * sd.C + c0 + c
                                              : static_cast<int64_t>(c0 + c) * p.R + j);
    if (!store_ok(p.status, j < p.R && c0 + c < sd.C)) continue;
    if constexpr (F32)
      static_cast<float *>(sd.out)[at] = f * s;
    else
      static_cast<__nv_bfloat16 *>(sd.out)[at] = __float2bfloat16_rn(f * s);
  }
  if (shares > 1) cluster.sync();
}

// ------------------------------------------------------------------ host side
int sm_count() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 148;
}

// Launch with dynamic shared memory and clusters of `cluster` blocks along the
// grid's dimension `dim` (0 x, 1 y, 2 z).
template <auto Kernel, typename Args>
cudaError_t launch(dim3 grid, int smem, int cluster, int dim, const Args &args,
                   cudaStream_t stream) {
  static bool attr_set[64] = {};  // per kernel and device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = dim == 0 ? cluster : 1;
  attr[0].val.clusterDim.y = dim == 1 ? cluster : 1;
  attr[0].val.clusterDim.z = dim == 2 ? cluster : 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, Kernel, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int RT, bool TRANS>
cudaError_t run_contract(const ContractArgs &a, cudaStream_t stream) {
  // Slices of the contracted dimension: enough blocks for two per SM, none
  // shorter than 256 columns.
  const int64_t tiles = plan_max_tiles(a.M, a.L);
  int slices = 1;
  while (slices < 8 && tiles * slices < 2 * sm_count() && a.C >= 256 * slices * 2) slices *= 2;
  return launch<lora_contract_kernel<RT, TRANS>>(dim3(static_cast<unsigned>(tiles), slices),
                                                 ContractSmem<RT, TRANS>::kBytes, slices, 1, a,
                                                 stream);
}

template <int RT, bool TRANS, bool F32>
cudaError_t run_expand(const ExpandArgs &a, cudaStream_t stream) {
  const int64_t tiles = plan_max_tiles(a.M, a.L);
  const int64_t blocks = tiles * ((a.C + kSlab - 1) / kSlab);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch<lora_expand_kernel<RT, TRANS, F32>>(dim3(static_cast<unsigned>(blocks)),
                                                    ExpandSmem<RT, TRANS, F32>::kBytes, 1, 0, a,
                                                    stream);
}

template <int RT, bool F32>
cudaError_t run_outer(const OuterArgs &a, cudaStream_t stream) {
  const int slabs = a.slabs0 + (a.side[1].C + 63) / 64;
  // Shares of an adapter's rows: enough blocks for four per SM, none with
  // fewer than two row tiles on average.
  int shares = 1;
  while (shares < 8 && static_cast<int64_t>(slabs) * a.L * shares < 4 * sm_count() &&
         a.M / a.L >= 2 * kTileRows * shares * 2)
    shares *= 2;
  return launch<lora_outer_kernel<RT, F32>>(dim3(slabs, a.L, shares), OuterSmem<RT, F32>::kBytes,
                                            shares, 2, a, stream);
}

template <typename F>
cudaError_t by_rank(int R, F &&f) {
  if (R <= 16) return f(std::integral_constant<int, 16>());
  if (R <= 32) return f(std::integral_constant<int, 32>());
  if (R <= 64) return f(std::integral_constant<int, 64>());
  return f(std::integral_constant<int, 128>());
}

}  // namespace

size_t lora_plan_words(int64_t M, int32_t L) {
  return static_cast<size_t>(plan_tiles_at(M, L) + 2 * plan_max_tiles(M, L));
}

cudaError_t launch_lora_plan(const int32_t *adapter, int64_t M, int32_t L, int32_t *plan,
                             int *status, cudaStream_t stream) {
  const int bytes = (kPlanWarps * (L + 1) + 2 * (L + 2)) * 4;
  cudaError_t e = cudaFuncSetAttribute(lora_plan_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  lora_plan_kernel<<<1, kPlanWarps * 32, bytes, stream>>>(adapter, static_cast<int32_t>(M), L,
                                                          plan, status);
  return cudaGetLastError();
}

cudaError_t launch_lora_forward(const LoraRequest &q, cudaStream_t stream) {
  const ContractArgs c = {q.x, q.ldx, q.A, nullptr, q.plan, q.t, q.M,
                          static_cast<int32_t>(q.K), q.R, q.L, q.status};
  const ExpandArgs e = {q.t, q.B, q.scale, q.plan, q.base, q.ld_base, q.y, q.ldy, q.M,
                        static_cast<int32_t>(q.N), q.R, q.L, q.status};
  return by_rank(q.R, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    const cudaError_t err = run_contract<RT, false>(c, stream);
    if (err != cudaSuccess) return err;
    return q.f32 ? run_expand<RT, false, true>(e, stream) : run_expand<RT, false, false>(e, stream);
  });
}

cudaError_t launch_lora_backward(const LoraRequest &q, cudaStream_t stream) {
  return by_rank(q.R, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    if (q.M > 0) {
      const ContractArgs c = {q.dy, q.lddy, q.B, q.scale, q.plan, q.dt, q.M,
                              static_cast<int32_t>(q.N), q.R, q.L, q.status};
      const cudaError_t err = run_contract<RT, true>(c, stream);
      if (err != cudaSuccess) return err;
    }
    if (q.dA != nullptr) {
      OuterArgs o = {};
      o.side[0] = {q.dy, q.lddy, q.t, q.scale, q.dB, static_cast<int32_t>(q.N), 0};
      o.side[1] = {q.x, q.ldx, q.dt, nullptr, q.dA, static_cast<int32_t>(q.K), 1};
      o.slabs0 = static_cast<int32_t>((q.N + 63) / 64);
      o.plan = q.plan;
      o.M = q.M;
      o.R = q.R;
      o.L = q.L;
      o.status = q.status;
      const cudaError_t err =
          q.f32 ? run_outer<RT, true>(o, stream) : run_outer<RT, false>(o, stream);
      if (err != cudaSuccess) return err;
    }
    if (q.M > 0 && q.dx != nullptr) {
      const ExpandArgs e = {q.dt, q.A, nullptr, q.plan, q.base, q.ld_base, q.dx, q.lddx, q.M,
                            static_cast<int32_t>(q.K), q.R, q.L, q.status};
      return run_expand<RT, true, false>(e, stream);
    }
    return cudaSuccess;
  });
}

}  // namespace sq
