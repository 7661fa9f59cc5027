// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   t[m] = A[a] x[m]                 (rank R)        y[m] = base[m] + c[a] B[a] t[m]
//   dt[m] = c[a] B[a]^T dy[m]                        dx[m] = dx_base[m] + A[a]^T dt[m]
//   dB[a] = c[a] sum_{m of a} dy[m] t[m]^T           dA[a] = sum_{m of a} dt[m] x[m]^T
//
// with a = adapter[m].  A plan, made once per batch, lists the rows adapter by
// adapter and cuts them into tiles of at most 128 rows of one adapter, so that
// every tile is an ordinary pair of thin matrix products whatever the order of
// the rows: scattered rows are gathered, single tokens of one adapter share a
// tile, and the plan serves every layer that the batch goes through.
//
// Three kernels:
//   contract  [rows] x [C] -> [rows] x R: t (rows of A) and dt (columns of B);
//   expand    [rows] x R -> [rows] x [C] added to base: y and dx;
//   outer     [rows] x [C], [rows] x R -> [C] x R: dB and dA.
// All are bound by the rows' traffic (at rank 64 a row element that is read
// and written, four bytes, meets 128 flop).  Sums are fp32; the small operand t
// (dt) enters the second product as bf16 where the result is rounded to bf16
// anyway, or split into three bf16 terms (24 significant bits) where the result
// stays fp32.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mma.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

namespace cg = cooperative_groups;

constexpr int kTileRows = SQ_LORA_TILE_ROWS;
constexpr int32_t kPlanMagic = 0x53514C32;

// ------------------------------------------------------------------- the plan
// int32 words: [0] magic, [1] M, [2] L, [3] tiles, tile_at[L + 2] (the first tile
// of each bin; bin L holds the rows without an adapter), padding to a multiple
// of four, then a record per tile: {bin, rows, first place in the order by
// adapter, 1 if its rows are neighbours, row numbers[128]}.  A kernel finds
// everything about its tile at one address; row numbers past the tile's rows
// repeat its first.
constexpr int kRecWords = 4 + kTileRows;
__host__ __device__ inline int64_t plan_recs_at(int32_t L) { return (4 + (L + 2) + 3) / 4 * 4; }
__host__ __device__ inline int64_t plan_max_tiles(int64_t M, int32_t L) {
  return M / kTileRows + (M < L + 1 ? M : L + 1);
}
// A plan of another batch size or adapter count: reported, nothing computed.
__device__ __forceinline__ bool plan_fits(const int32_t *plan, int64_t M, int32_t L,
                                          int *status) {
  const int4 h = *reinterpret_cast<const int4 *>(plan);
  const bool ok = h.x == kPlanMagic && h.y == static_cast<int32_t>(M) && h.z == L;
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
    if (store_ok(status, threadIdx.x < plan_recs_at(L))) plan[threadIdx.x] = v[threadIdx.x];
  }
  for (int b = threadIdx.x; b <= bins; b += blockDim.x)
    if (store_ok(status, 4 + b < plan_recs_at(L))) plan[4 + b] = tile_at[b];
  int32_t *recs = plan + plan_recs_at(L);
  const int64_t max_tiles = plan_max_tiles(M, L);
  for (int b = warp; b < bins; b += kPlanWarps)
    for (int i = lane; i < tile_at[b + 1] - tile_at[b]; i += 32) {
      const int64_t at = tile_at[b] + i;
      if (!store_ok(status, at < max_tiles)) continue;
      const int first = start[b] + i * kTileRows, left = start[b + 1] - first;
      recs[at * kRecWords] = b;
      recs[at * kRecWords + 1] = left < kTileRows ? left : kTileRows;
      recs[at * kRecWords + 2] = first;
    }
  // places: 32 rows a step in order; equal bins of a step rank by lane
  for (int64_t r0 = lo; r0 < hi; r0 += 32) {
    const int64_t r = r0 + lane;
    const bool in = r < hi;
    const int32_t a = in ? adapter[r] : 0;
    const int b = !in ? -1 : (a >= 0 && a < L ? a : L);
    const unsigned same = __match_any_sync(~0u, b);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (in) {
      const int place = mine[b] + rank;  // within the bin
      const int64_t at = tile_at[b] + place / kTileRows;
      if (store_ok(status, at < max_tiles)) {
        int32_t *rows = recs + at * kRecWords + 4;
        rows[place % kTileRows] = static_cast<int32_t>(r);
        // the tile's first row also fills the places past its last
        if (place % kTileRows == 0) {
          const int left = start[b + 1] - start[b] - place;
          for (int i = left; i < kTileRows; ++i) rows[i] = static_cast<int32_t>(r);
        }
      }
    }
    __syncwarp();
    if (in && rank == 0) mine[b] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // rows ascend within a tile: neighbours if the last is the first + rows - 1
  for (int64_t at = threadIdx.x; at < tile_at[bins]; at += blockDim.x) {
    int32_t *rec = recs + at * kRecWords;
    if (store_ok(status, at < max_tiles)) rec[3] = rec[4 + rec[1] - 1] - rec[4] == rec[1] - 1;
  }
}

// ----------------------------------------------------------------- shared parts
// v as TERMS bf16 values whose sum has 8 TERMS significant bits, packed in pairs.
template <int TERMS>
__device__ __forceinline__ void split_terms(float4 v, uint2 (&out)[TERMS]) {
#pragma unroll
  for (int s = 0; s < TERMS; ++s) {
    const uint32_t lo = bf16x2(v.x, v.y), hi = bf16x2(v.z, v.w);
    out[s] = make_uint2(lo, hi);
    v = make_float4(v.x - bf16_lo(lo), v.y - bf16_hi(lo), v.z - bf16_lo(hi), v.w - bf16_hi(hi));
  }
}

// ------------------------------------------------------------------- contract
// out[m][j] = f sum_c in[m][c] W(j, c), f = scale[a] or 1; W(j, c) = w[a][j][c]
// (TRANS false: A) or w[a][c][j] (TRANS true: B, an operand whose rows run
// along the contraction).  One block per row tile and slice of the contracted
// dimension: TMA brings the tile's rows, 64 columns a stage -- one box where
// they are neighbours, four rows by number at a time where they are scattered
// (110 MB of rows: 43 us against 72) -- and the weight's box beside them; one
// thread issues tcgen05.mma (M = 128, N = RT, sums in tensor memory), so that
// reading the rows costs the SM no instructions.  The blocks of a cluster hold the slices of one tile and add
// their partial sums through distributed shared memory in a fixed order.  The
// forward pass stores t by row in fp32; the backward pass stores dt, and beside
// it t, as bf16 terms by tile, 128 rows each with zeros past the tile's last:
// the operand that the outer products and dx read.
struct ContractArgs {
  const float *scale;  // nullptr: 1
  const int32_t *plan;
  float *out;             // forward: t [M][R]
  const float *t;         // backward: t [M][R]
  uint16_t *vt, *vdt;     // backward: [TERMS][max_tiles][128][R]
  int64_t M, max_tiles;
  int32_t C, R, L;
  int *status;
};

constexpr int kContractThreads = 128;

template <int RT>
struct ContractSmem {
  static constexpr int kStages = RT == 64 ? 4 : 3;
  static constexpr int kIn = kTileRows * 128;
  static constexpr int kW = RT * 128;  // both orders: 64 columns by RT
  static constexpr int kStage = kIn + kW;
  static constexpr int kBars = kStages * kStage;
  static constexpr int kBytes = kBars + (2 * kStages + 1) * 8 + 16 + 1024;
  static constexpr int kPartRow = RT + 4;  // floats
  static_assert(kTileRows * kPartRow * 4 <= kBars, "partial sums reuse the stages");
};

// TERMS 0: the forward pass.
template <int RT, bool TRANS, int TERMS>
__global__ void __launch_bounds__(kContractThreads)
    lora_contract_kernel(const __grid_constant__ CUtensorMap tm_in,
                         const __grid_constant__ CUtensorMap tm_rows,
                         const __grid_constant__ CUtensorMap tm_w, const ContractArgs p) {
  using S = ContractSmem<RT>;
  constexpr int STAGES = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *empty = full + STAGES;
  uint64_t *done = empty + STAGES;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int slices = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_in);
    prefetch_tmap(&tm_rows);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, RT);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_dependency_launch();

  // A fitting plan has a record for every block of the grid; the blocks of a
  // cluster share their tile and so their way through this kernel.
  int4 tile = make_int4(p.L, 0, 0, 0);
  const int32_t *rec = p.plan + plan_recs_at(p.L) + static_cast<int64_t>(blockIdx.x) * kRecWords;
  if (plan_fits(p.plan, p.M, p.L, p.status) && static_cast<int>(blockIdx.x) < p.plan[3])
    tile = *reinterpret_cast<const int4 *>(rec);
  const int bin = tile.x, count = tile.y;
  if (bin < p.L) {
    const int slice = ((p.C + slices - 1) / slices + 63) / 64 * 64;
    const int c_lo = rank * slice;
    const int c_hi = c_lo + slice < p.C ? c_lo + slice : p.C;
    const int steps = c_hi > c_lo ? (c_hi - c_lo + 63) / 64 : 0;
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      // Scattered: lane l brings rows 4 l .. 4 l + 3; groups past the tile's
      // last row are left out.  Whatever stands in a row past the last only
      // meets sums that are not stored.
      const bool run = tile.w != 0;
      const bool brings = !run && 4 * lane < count;
      const int4 rows = *reinterpret_cast<const int4 *>(rec + 4 + 4 * lane);
      const uint32_t bytes = (run ? S::kIn : (count + 3) / 4 * 512) + S::kW;
      uint32_t armed = 0, armed_parity = 0;
      for (int step = 0; step < steps; ++step) {
        const int st = step % STAGES;
        const uint32_t phase = (step / STAGES) & 1;
        bool ok = true;
        uint8_t *in = smem + st * S::kStage;
        const int c0 = c_lo + step * 64;
        if (lane == 0) {
          ok = bounded_wait(&empty[st], phase ^ 1, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT);
          if (ok) {
            mbar_arrive_expect_tx(&full[st], bytes);
            if (run) tma_load_2d(in, &tm_in, &full[st], c0, rows.x);
            if constexpr (!TRANS) {
              tma_load_3d(in + S::kIn, &tm_w, &full[st], c0, 0, bin);
            } else {
#pragma unroll
              for (int h = 0; h < RT / 64; ++h)
                tma_load_3d(in + S::kIn + h * 8192, &tm_w, &full[st], h * 64, c0, bin);
            }
            armed |= 1u << st;
            armed_parity = (armed_parity & ~(1u << st)) | (phase << st);
          }
        }
        if (!__shfl_sync(~0u, ok, 0)) break;
        if (brings) tma_gather4(in + lane * 512, &tm_rows, &full[st], c0, rows);
        __syncwarp();
      }
      // never leave with a copy in flight into this block's shared memory
      if (lane == 0)
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s)) mbar_wait(&full[s], (armed_parity >> s) & 1u, kBoundedWaitNs);
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_bf16(kTileRows, RT) | (TRANS ? kIdescTransB : 0u);
        for (int step = 0; step < steps; ++step) {
          const int st = step % STAGES;
          if (!bounded_wait(&full[st], (step / STAGES) & 1, abort_flag, p.status,
                            SQ_ERR_DEVICE_TIMEOUT))
            break;
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + st * S::kStage), sb = sa + S::kIn;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_tc(tmem, sdesc_kmajor_sw128(sa + kk * 32),
                        TRANS ? sdesc_mnmajor_sw128(sb + kk * 2048, 8192)
                              : sdesc_kmajor_sw128(sb + kk * 32),
                        idesc, (step | kk) != 0);
          mma_commit(&empty[st]);
        }
        mma_commit(done);
      }
      __syncwarp();
    }
    const bool ok = bounded_wait(done, 0, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT);
    tc_fence_after();
    // nothing reads or fills the stages any more
    __syncthreads();

    // partial sums -> shared memory -> sum over the slices
    float *part = reinterpret_cast<float *>(smem);
    constexpr int PS = S::kPartRow;
#pragma unroll
    for (int c = 0; c < RT; c += 32) {
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(tmem + c + (static_cast<uint32_t>(warp * 32) << 16), r);
      tmem_ld_wait();
      float *to = part + threadIdx.x * PS + c;
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<uint4 *>(to + j) =
            steps > 0 ? make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]) : make_uint4(0, 0, 0, 0);
    }
    if (slices > 1) cluster.sync(); else __syncthreads();
    const float f = p.scale ? p.scale[bin] : 1.0f;
    const int quads = p.R / 4;
    const int total = ok ? (TERMS > 0 ? kTileRows : count) * quads : 0;
    for (int e = rank * kContractThreads + threadIdx.x; e < total;
         e += slices * kContractThreads) {
      const int r = e / quads, j = (e - r * quads) * 4;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (TERMS == 0 || r < count) {
        for (int q = 0; q < slices; ++q) {
          const float *src = slices > 1 ? cluster.map_shared_rank(part, q) : part;
          const float4 v = *reinterpret_cast<const float4 *>(src + r * PS + j);
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
        s = make_float4(f * s.x, f * s.y, f * s.z, f * s.w);
      }
      const int row = rec[4 + r];
      const int64_t at = static_cast<int64_t>(row) * p.R + j;
      if constexpr (TERMS == 0) {
        if (store_ok(p.status, row >= 0 && row < p.M))
          *reinterpret_cast<float4 *>(p.out + at) = s;
      } else {
        const int64_t place = static_cast<int64_t>(blockIdx.x) * kTileRows + r;
        if (!store_ok(p.status, place < p.max_tiles * kTileRows)) continue;
        float4 tv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < count) tv = *reinterpret_cast<const float4 *>(p.t + at);
        uint2 d[TERMS], t[TERMS];
        split_terms<TERMS>(s, d);
        split_terms<TERMS>(tv, t);
#pragma unroll
        for (int q = 0; q < TERMS; ++q) {
          const int64_t to = (q * p.max_tiles * kTileRows + place) * p.R + j;
          *reinterpret_cast<uint2 *>(p.vdt + to) = d[q];
          *reinterpret_cast<uint2 *>(p.vt + to) = t[q];
        }
      }
    }
    if (slices > 1) cluster.sync();  // no block leaves while its sums are read
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, RT);
  }
}

// --------------------------------------------------------------------- expand
// out[m][c] = base[m][c] + f sum_j t[m][j] W(j, c); W(j, c) = w[a][c][j] (TRANS
// false: B, t fp32 by row) or w[a][j][c] (TRANS true: A, t bf16 by tile).
// Persistent blocks, one per SM, take equal shares of the units (row tile, slab
// of 128 columns), neighbouring slabs of a tile in a row, so that t is loaded
// once for many slabs.  Every thread copies the pieces of base that it will
// add to, 16 bytes each, asynchronously into slots of its own some units ahead
// (nobody else reads them, so they need no barrier), and writes its sums back
// in 16-byte pieces: the columns of a slab are dealt to the product's columns
// so that the eight that a thread holds of a row in four accumulator tiles are
// neighbours.  Column 32 b + 8 c + 2 j + e is
// column 2 c + e of tile 4 b + j; the weight slab is permuted accordingly on
// its way into shared memory.  Rows without an adapter are copied from base
// (left alone when out is base).
struct ExpandArgs {
  const float *t;      // TRANS false: [M][R]
  const uint16_t *vt;  // TRANS true: [max_tiles][128][R]
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

constexpr int kExpandThreads = 512;

template <int RT, bool TRANS, bool F32>
struct ExpandSmem {
  static constexpr int kTerms = F32 ? 3 : 1;  // bf16 terms of t
  static constexpr int kSlab = F32 || RT > 64 ? 64 : 128;  // columns of a unit
  static constexpr int kTRow = RT * 2 + 16;
  static constexpr int kT = kTerms * kTileRows * kTRow;
  static constexpr int kWRow = TRANS ? kSlab * 2 + 16 : RT * 2 + 16;
  static constexpr int kW = TRANS ? RT * kWRow : kSlab * kWRow;
  static constexpr int kPieces = kTileRows * kSlab * (F32 ? 4 : 2) / 16 / kExpandThreads;
  static constexpr int kBase = kPieces * kExpandThreads * 16;
  static constexpr int kStage = kW + kBase;
  static constexpr int kFit = (224 * 1024 - kT) / kStage;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kBytes = kT + kStages * kStage;
  static_assert(kStages >= 2, "one unit ahead at least");
  static_assert(kBytes <= 232448, "dynamic shared memory above the per-block limit");
};

template <int RT, bool TRANS, bool F32>
__global__ void __launch_bounds__(kExpandThreads) lora_expand_kernel(const ExpandArgs p) {
  using S = ExpandSmem<RT, TRANS, F32>;
  constexpr int E = F32 ? 4 : 2;
  constexpr int Q = F32 ? 2 : 1;       // 16-byte pieces of eight columns
  constexpr int SLAB = S::kSlab;
  constexpr int NB = SLAB / 64;        // blocks of 32 columns of a warp
  constexpr int KK = RT / 16;
  static_assert(S::kPieces == 2 * NB * Q, "a thread's share of a unit");
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = warp & 7, wn = warp >> 3;  // 16 rows, half of the slab
  const int g = lane >> 2, c8 = (lane & 3) * 8;

  // base, weights and plan were complete before the kernel ahead of this one
  // began; only its own output, t, has to be waited for
  const int32_t *recs = p.plan + plan_recs_at(p.L);
  const int slabs = (p.C + SLAB - 1) / SLAB;
  const bool fits = plan_fits(p.plan, p.M, p.L, p.status);
  const int tiles = fits ? p.plan[3] : 0;
  const int64_t units = static_cast<int64_t>(tiles) * slabs;
  const int64_t u_lo = units * blockIdx.x / gridDim.x;
  const int mine = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - u_lo);
  const bool in_place = p.base == p.out;
  const int tile0 = static_cast<int>(u_lo / slabs), slab0 = static_cast<int>(u_lo % slabs);

  // A unit's weights and base -> its stage.  The thread's rows of base are
  // wm 16 + g (+ 8), its columns wn SLAB/2 + 32 b + c8 .. + 7.
  int l_tile = tile0, l_slab = slab0, l_bin = 0, l_count = 0;
  int32_t l_row[2] = {0, 0};
  auto next_tile = [&]() {
    const int32_t *rec = recs + static_cast<int64_t>(l_tile) * kRecWords;
    l_bin = rec[0];
    l_count = rec[1];
    l_row[0] = rec[4 + wm * 16 + g];
    l_row[1] = rec[4 + wm * 16 + g + 8];
  };
  auto load = [&](int stage) {
    const uint32_t sw = sm + S::kT + stage * S::kStage;
    const int c0 = l_slab * SLAB;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int col = c0 + wn * (SLAB / 2) + b * 32 + c8;
        const bool ok = p.base != nullptr && wm * 16 + g + h * 8 < l_count && col < p.C;
        const uint8_t *src = static_cast<const uint8_t *>(p.base) +
                             (l_row[h] * p.ld_base + col) * E;
#pragma unroll
        for (int q = 0; q < Q; ++q)
          cp_async16(sw + S::kW + (((h * NB + b) * Q + q) * kExpandThreads + tid) * 16,
                     ok ? src + q * 16 : reinterpret_cast<const uint8_t *>(p.w), ok);
      }
    if (l_bin < p.L) {
      const uint16_t *w = p.w + static_cast<int64_t>(l_bin) * p.R * p.C;
      if constexpr (!TRANS) {
        constexpr int PER = RT / 8;
#pragma unroll
        for (int k = tid; k < SLAB * PER; k += kExpandThreads) {
          const int r = k / PER, cc = k % PER;
          const int at = (r & ~31) | (((r >> 1) & 3) << 3) | (((r >> 3) & 3) << 1) | (r & 1);
          const bool ok = c0 + r < p.C && cc * 8 < p.R;
          cp_async16(sw + at * S::kWRow + cc * 16,
                     ok ? w + static_cast<int64_t>(c0 + r) * p.R + cc * 8 : w, ok);
        }
      } else {
        constexpr int PER = SLAB / 2;  // pairs of columns
#pragma unroll 8
        for (int k = tid; k < RT * PER; k += kExpandThreads) {
          const int r = k / PER, cc = k % PER;
          const int at = (cc & ~15) | ((cc & 3) << 2) | ((cc >> 2) & 3);
          const bool ok = r < p.R && c0 + cc * 2 < p.C;
          cp_async4(sw + r * S::kWRow + at * 4,
                    ok ? w + static_cast<int64_t>(r) * p.C + c0 + cc * 2 : w, ok);
        }
      }
    }
    if (++l_slab == slabs) {
      l_slab = 0;
      if (++l_tile < tiles) next_tile();
    }
  };

  if (mine > 0) next_tile();
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (s < mine) load(s);
    cp_async_commit();
  }
  grid_dependency_wait();

  int tile = tile0, slab = slab0, bin = 0, count = 0, stage = 0;
  int32_t row[2] = {0, 0};
  float f = 1.0f;
  bool fresh = true;
  for (int i = 0; i < mine; ++i) {
    if (fresh) {
      const int32_t *rec = recs + static_cast<int64_t>(tile) * kRecWords;
      bin = rec[0];
      count = rec[1];
      row[0] = rec[4 + wm * 16 + g];
      row[1] = rec[4 + wm * 16 + g + 8];
      if (i > 0) __syncthreads();  // the last tile's t is no longer read
      if (bin < p.L) {
        f = p.scale ? p.scale[bin] : 1.0f;
        if constexpr (TRANS) {
          for (int k = tid; k < kTileRows * (RT / 8); k += kExpandThreads) {
            const int r = k / (RT / 8), cc = k % (RT / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (cc * 8 < p.R)
              v = *reinterpret_cast<const uint4 *>(
                  p.vt + (static_cast<int64_t>(tile) * kTileRows + r) * p.R + cc * 8);
            *reinterpret_cast<uint4 *>(smem + r * S::kTRow + cc * 16) = v;
          }
        } else {
          for (int k = tid; k < kTileRows * (RT / 4); k += kExpandThreads) {
            const int r = k / (RT / 4), cc = k % (RT / 4);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < count && cc * 4 < p.R)
              v = *reinterpret_cast<const float4 *>(
                  p.t + static_cast<int64_t>(rec[4 + r]) * p.R + cc * 4);
            uint2 o[S::kTerms];
            split_terms<S::kTerms>(v, o);
#pragma unroll
            for (int s = 0; s < S::kTerms; ++s)
              *reinterpret_cast<uint2 *>(smem + (s * kTileRows + r) * S::kTRow + cc * 8) = o[s];
          }
        }
      }
    }
    cp_async_wait<S::kStages - 2>();
    __syncthreads();
    if (i + S::kStages - 1 < mine) load(stage == 0 ? S::kStages - 1 : stage - 1);
    cp_async_commit();
    if (wm * 16 < count && (bin < p.L || !in_place)) {
      const uint8_t *st = smem + S::kT + stage * S::kStage;
      float acc[4 * NB][4];
#pragma unroll
      for (int n = 0; n < 4 * NB; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[n][k] = 0.0f;
      if (bin < p.L) {
        const uint32_t sw = smem_u32(st);
#pragma unroll 1
        for (int s = S::kTerms - 1; s >= 0; --s) {  // the smallest terms first
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) {
            uint32_t a[4];
            ldsm_x4(sm + (s * kTileRows + wm * 16 + (lane & 15)) * S::kTRow +
                        (kk * 16 + (lane >> 4) * 8) * 2,
                    a);
#pragma unroll
            for (int n = 0; n < 4 * NB; n += 2) {
              uint32_t b[4];
              const int col = wn * (SLAB / 2) + n * 8;
              if constexpr (!TRANS)
                ldsm_x4(sw + (col + (lane & 7) + ((lane >> 4) << 3)) * S::kWRow +
                            (kk * 16 + ((lane >> 3) & 1) * 8) * 2,
                        b);
              else
                ldsm_x4_t(sw + (kk * 16 + (lane & 15)) * S::kWRow + (col + (lane >> 4) * 8) * 2,
                          b);
              mma_bf16(acc[n], a, b[0], b[1]);
              mma_bf16(acc[n + 1], a, b[2], b[3]);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (wm * 16 + g + h * 8 >= count) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int col = slab * SLAB + wn * (SLAB / 2) + b * 32 + c8;
          if (col >= p.C || !store_ok(p.status, row[h] >= 0 && row[h] < p.M && col + 8 <= p.ld_out))
            continue;
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) +
                                                 (row[h] * p.ld_out + col) * E);
          uint32_t o[4 * Q];
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const uint4 v = *reinterpret_cast<const uint4 *>(
                st + S::kW + (((h * NB + b) * Q + q) * kExpandThreads + tid) * 16);
            o[4 * q] = v.x;
            o[4 * q + 1] = v.y;
            o[4 * q + 2] = v.z;
            o[4 * q + 3] = v.w;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = acc[b * 4 + j][2 * h], y = acc[b * 4 + j][2 * h + 1];
            if constexpr (F32) {
              o[2 * j] = __float_as_uint(fmaf(f, x, __uint_as_float(o[2 * j])));
              o[2 * j + 1] = __float_as_uint(fmaf(f, y, __uint_as_float(o[2 * j + 1])));
            } else {
              o[j] = bf16x2(fmaf(f, x, bf16_lo(o[j])), fmaf(f, y, bf16_hi(o[j])));
            }
          }
#pragma unroll
          for (int q = 0; q < Q; ++q)
            dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
    }
    if (++stage == S::kStages) stage = 0;
    fresh = ++slab == slabs;
    if (fresh) {
      slab = 0;
      ++tile;
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------- outer
// out[a](c, j) = f sum_{m of a} src[m][c] v[m][j]: dB[a][n][j] (src dy, v t, f =
// scale) and dA[a][j][k] (src x, v dt, f = 1, stored transposed).  One block
// per adapter, slab of 128 columns c and share of the adapter's rows, 64 rows a
// stage: TMA brings src's rows -- as a box where 64 neighbours are the
// adapter's, else by number -- and v's box; both are operands whose rows run
// along the contraction, M = 128 columns of src by N = RT.  v is zero in the
// rows past a tile's last, where src repeats a row of the tile.  The
// blocks of a cluster hold the shares and add them in a fixed order.  Rows are
// taken from the last to the first: dy's last rows are what the contraction
// before left in L2.
struct OuterSide {
  const float *scale;  // nullptr: 1
  void *out;
  int32_t C;
  int32_t transposed;  // out [R][C] instead of [C][R]
};
struct OuterArgs {
  OuterSide side[2];
  int32_t slabs0;  // slabs of side 0
  const int32_t *plan;
  int64_t M, max_tiles;
  int32_t R, L;
  int *status;
};
struct OuterMaps {
  CUtensorMap src[2], rows[2], v[2];
};

constexpr int kOuterThreads = 128;
constexpr int kOuterSlab = 128;
constexpr int kOuterRows = 64;  // a stage

template <int RT, int TERMS>
struct OuterSmem {
  static constexpr int kSrc = kOuterRows * kOuterSlab * 2;  // two boxes of 64 columns
  static constexpr int kV = TERMS * kOuterRows * RT * 2;
  static constexpr int kStage = kSrc + kV;
  static constexpr int kStages = 4 * kStage <= 104 * 1024 ? 4 : 3;
  static constexpr int kBars = kStages * kStage;
  static constexpr int kPartRow = RT + 1;  // floats
  static constexpr int kBytes = kBars + (2 * kStages + 1) * 8 + 16 + 1024;
  static_assert(kOuterSlab * kPartRow * 4 <= kBars, "partial sums reuse the stages");
  static_assert(kBytes <= 232448, "dynamic shared memory above the per-block limit");
};

template <int RT, int TERMS>
__global__ void __launch_bounds__(kOuterThreads)
    lora_outer_kernel(const __grid_constant__ OuterMaps maps, const OuterArgs p) {
  using S = OuterSmem<RT, TERMS>;
  constexpr int STAGES = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *empty = full + STAGES;
  uint64_t *done = empty + STAGES;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int shares = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool second = static_cast<int>(blockIdx.x) >= p.slabs0;
  const OuterSide sd = second ? p.side[1] : p.side[0];
  const CUtensorMap *tm_src = second ? &maps.src[1] : &maps.src[0];
  const CUtensorMap *tm_rows = second ? &maps.rows[1] : &maps.rows[0];
  const CUtensorMap *tm_v = second ? &maps.v[1] : &maps.v[0];
  const int c0 = (static_cast<int>(blockIdx.x) - (second ? p.slabs0 : 0)) * kOuterSlab;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(tm_src);
    prefetch_tmap(tm_rows);
    prefetch_tmap(tm_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, RT);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int bin = blockIdx.y;
  const bool fits = plan_fits(p.plan, p.M, p.L, p.status);
  int tile0 = 0, steps = 0, all = 0;
  const int32_t *recs = p.plan + plan_recs_at(p.L);
  if (fits) {
    tile0 = p.plan[4 + bin];
    const int tiles = p.plan[4 + bin + 1] - tile0;
    // stages of 64 rows: two per full tile, one or two in the last
    if (tiles > 0)
      all = 2 * (tiles - 1) +
            (recs[static_cast<int64_t>(tile0 + tiles - 1) * kRecWords + 1] + kOuterRows - 1) /
                kOuterRows;
    steps = all > rank ? (all - rank + shares - 1) / shares : 0;
  }
  grid_dependency_wait();

  if (fits) {
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      // lane l: rows 4 (l % 16) .. + 3 of column box l / 16
      const bool brings = c0 + (lane >> 4) * 64 < sd.C;  // no box past the last column
      const uint32_t bytes = S::kV + (c0 + 64 < sd.C ? 2 : 1) * 8192;
      uint32_t armed = 0, armed_parity = 0;
      int4 rows = make_int4(0, 0, 0, 0);
      bool run = false;
      auto fetch = [&](int step) {
        const int s64 = all - 1 - (rank + step * shares);
        const int32_t *rec = recs + static_cast<int64_t>(tile0 + s64 / 2) * kRecWords;
        rows = *reinterpret_cast<const int4 *>(rec + 4 + (s64 & 1) * 64 + (lane & 15) * 4);
        run = rec[3] != 0 && (s64 & 1) * 64 + kOuterRows <= rec[1];
      };
      if (steps > 0) fetch(0);
      for (int step = 0; step < steps; ++step) {
        const int st = step % STAGES;
        const uint32_t phase = (step / STAGES) & 1;
        const int s64 = all - 1 - (rank + step * shares);
        uint8_t *src = smem + st * S::kStage;
        bool ok = true;
        if (lane == 0) {
          ok = bounded_wait(&empty[st], phase ^ 1, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT);
          if (ok) {
            mbar_arrive_expect_tx(&full[st], bytes);
            if (run) {
              tma_load_2d(src, tm_src, &full[st], c0, rows.x);
              if (c0 + 64 < sd.C) tma_load_2d(src + 8192, tm_src, &full[st], c0 + 64, rows.x);
            }
            const int vrow = tile0 * kTileRows + s64 * kOuterRows;
#pragma unroll
            for (int q = 0; q < TERMS; ++q)
#pragma unroll
              for (int h = 0; h < RT / 64; ++h)
                tma_load_3d(src + S::kSrc + (q * (RT / 64) + h) * 8192, tm_v, &full[st], h * 64,
                            vrow, q);
            armed |= 1u << st;
            armed_parity = (armed_parity & ~(1u << st)) | (phase << st);
          }
        }
        if (!__shfl_sync(~0u, ok, 0)) break;
        if (brings && !run)
          tma_gather4(src + (lane >> 4) * 8192 + (lane & 15) * 512, tm_rows, &full[st],
                      c0 + (lane >> 4) * 64, rows);
        if (step + 1 < steps) fetch(step + 1);
        __syncwarp();
      }
      if (lane == 0)
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s)) mbar_wait(&full[s], (armed_parity >> s) & 1u, kBoundedWaitNs);
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_bf16(kOuterSlab, RT) | kIdescTransA | kIdescTransB;
        for (int step = 0; step < steps; ++step) {
          const int st = step % STAGES;
          if (!bounded_wait(&full[st], (step / STAGES) & 1, abort_flag, p.status,
                            SQ_ERR_DEVICE_TIMEOUT))
            break;
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + st * S::kStage), sb = sa + S::kSrc;
#pragma unroll
          for (int q = TERMS - 1; q >= 0; --q)
#pragma unroll
            for (int kk = 0; kk < kOuterRows / 16; ++kk)
              mma_bf16_tc(tmem, sdesc_mnmajor_sw128(sa + kk * 2048, 8192),
                          sdesc_mnmajor_sw128(sb + q * (RT / 64) * 8192 + kk * 2048, 8192), idesc,
                          step > 0 || kk > 0 || q < TERMS - 1);
          mma_commit(&empty[st]);
        }
        mma_commit(done);
      }
      __syncwarp();
    }
    const bool ok = bounded_wait(done, 0, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT);
    tc_fence_after();
    __syncthreads();  // nothing reads or fills the stages any more

    float *part = reinterpret_cast<float *>(smem);
    constexpr int PS = S::kPartRow;
#pragma unroll
    for (int c = 0; c < RT; c += 32) {
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(tmem + c + (static_cast<uint32_t>(warp * 32) << 16), r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        part[threadIdx.x * PS + c + j] = steps > 0 ? __uint_as_float(r[j]) : 0.0f;
    }
    if (shares > 1) cluster.sync(); else __syncthreads();
    const float f = sd.scale ? sd.scale[bin] : 1.0f;
    const int cols = sd.C - c0 < kOuterSlab ? sd.C - c0 : kOuterSlab;
    const int n_out = ok ? cols * p.R : 0;
    const int64_t obase = static_cast<int64_t>(bin) * p.R * sd.C;
    for (int e = rank * kOuterThreads + threadIdx.x; e < n_out; e += shares * kOuterThreads) {
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
      if constexpr (TERMS > 1)
        static_cast<float *>(sd.out)[at] = f * s;
      else
        static_cast<__nv_bfloat16 *>(sd.out)[at] = __float2bfloat16_rn(f * s);
    }
    if (shares > 1) cluster.sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, RT);
  }
}

// ------------------------------------------------------------------ host side
// Launch with dynamic shared memory and clusters of `cluster` blocks along the
// grid's dimension `dim` (0 x, 1 y, 2 z).  Every kernel here waits for the one
// ahead of it in the stream (programmatic dependent launch) before it reads
// what that one may have written.
template <auto Kernel, typename... Args>
cudaError_t launch(dim3 grid, int threads, int smem, int cluster, int dim, cudaStream_t stream,
                   const Args &...args) {
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
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = dim == 0 ? cluster : 1;
  attr[1].val.clusterDim.y = dim == 1 ? cluster : 1;
  attr[1].val.clusterDim.z = dim == 2 ? cluster : 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, Kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Tensor map of bf16 [d2][d1][d0] with row stride ld (elements), boxes of 64
// columns by `rows`, 128-byte swizzle; d2 == 0: two dimensions.
cudaError_t bf16_map(CUtensorMap *map, const void *ptr, int64_t d0, int64_t d1, int64_t d2,
                     int64_t ld, int rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1),
                              static_cast<cuuint64_t>(d2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2,
                                 static_cast<cuuint64_t>(ld) * 2 * static_cast<cuuint64_t>(d1)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 == 0 ? 2 : 3, const_cast<void *>(ptr),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int RT, bool TRANS, int TERMS>
cudaError_t run_contract(const uint16_t *in, int64_t ld, const uint16_t *w, const ContractArgs &a,
                         cudaStream_t stream) {
  CUtensorMap tm_in, tm_rows, tm_w;
  cudaError_t e = bf16_map(&tm_in, in, a.C, a.M, 0, ld, kTileRows);
  if (e == cudaSuccess) e = bf16_map(&tm_rows, in, a.C, a.M, 0, ld, 1);
  if (e == cudaSuccess)
    e = TRANS ? bf16_map(&tm_w, w, a.R, a.C, a.L, a.R, 64)
              : bf16_map(&tm_w, w, a.C, a.R, a.L, a.C, RT);
  if (e != cudaSuccess) return e;
  // Slices of the contracted dimension: as many blocks as run at once (two per
  // SM), none shorter than 256 columns.
  int slices = 1;
  while (slices < 8 && a.max_tiles * slices * 2 <= 2 * sm_count() && a.C >= 256 * slices * 2)
    slices *= 2;
  return launch<lora_contract_kernel<RT, TRANS, TERMS>>(
      dim3(static_cast<unsigned>(a.max_tiles), slices), kContractThreads,
      ContractSmem<RT>::kBytes, slices, 1, stream, tm_in, tm_rows, tm_w, a);
}

template <int RT, bool TRANS, bool F32>
cudaError_t run_expand(const ExpandArgs &a, cudaStream_t stream) {
  using S = ExpandSmem<RT, TRANS, F32>;
  const int64_t units = plan_max_tiles(a.M, a.L) * ((a.C + S::kSlab - 1) / S::kSlab);
  const int sms = sm_count();
  return launch<lora_expand_kernel<RT, TRANS, F32>>(
      dim3(static_cast<unsigned>(units < sms ? units : sms)), kExpandThreads, S::kBytes, 1, 0,
      stream, a);
}

template <int RT, int TERMS>
cudaError_t run_outer(const OuterMaps &maps, const OuterArgs &a, cudaStream_t stream) {
  const int slabs = a.slabs0 + (a.side[1].C + kOuterSlab - 1) / kOuterSlab;
  // Shares of an adapter's rows: as many blocks as run at once (two per SM),
  // none with fewer than two stages on average.
  int shares = 1;
  while (shares < 8 && static_cast<int64_t>(slabs) * a.L * shares * 2 <= 2 * sm_count() &&
         a.M / a.L >= 2 * kOuterRows * shares * 2)
    shares *= 2;
  return launch<lora_outer_kernel<RT, TERMS>>(dim3(slabs, a.L, shares), kOuterThreads,
                                              OuterSmem<RT, TERMS>::kBytes, shares, 2, stream,
                                              maps, a);
}

// Ranks are padded to 64 (128) columns: the boxes' columns past R read as zero.
template <typename F>
cudaError_t by_rank(int R, F &&f) {
  if (R <= 64) return f(std::integral_constant<int, 64>());
  return f(std::integral_constant<int, 128>());
}
// The expansion's inner dimension, in which padding costs products.
template <typename F>
cudaError_t by_rank_fine(int R, F &&f) {
  if (R <= 16) return f(std::integral_constant<int, 16>());
  if (R <= 32) return f(std::integral_constant<int, 32>());
  return by_rank(R, f);
}

template <int TERMS>
cudaError_t run_backward(const LoraRequest &q, cudaStream_t stream) {
  if (q.M == 0) {
    const size_t elem = TERMS > 1 ? 4 : 2, rank = static_cast<size_t>(q.L) * q.R;
    const cudaError_t err = cudaMemsetAsync(q.dA, 0, rank * q.K * elem, stream);
    return err != cudaSuccess ? err : cudaMemsetAsync(q.dB, 0, rank * q.N * elem, stream);
  }
  const int32_t N = static_cast<int32_t>(q.N), K = static_cast<int32_t>(q.K);
  const int64_t max_tiles = plan_max_tiles(q.M, q.L), rows = max_tiles * kTileRows;
  uint16_t *vdt = static_cast<uint16_t *>(q.workspace);
  uint16_t *vt = vdt + TERMS * rows * q.R;
  const ContractArgs c = {q.scale, q.plan, nullptr, q.t, vt,  vdt,
                          q.M,     max_tiles, N,    q.R, q.L, q.status};
  cudaError_t e = by_rank(q.R, [&](auto rt) {
    return run_contract<decltype(rt)::value, true, TERMS>(q.dy, q.lddy, q.B, c, stream);
  });
  if (e == cudaSuccess && q.dA != nullptr) {
    OuterMaps maps;
    OuterArgs o = {};
    o.side[0] = {q.scale, q.dB, N, 0};
    o.side[1] = {nullptr, q.dA, K, 1};
    o.slabs0 = (N + kOuterSlab - 1) / kOuterSlab;
    o.plan = q.plan;
    o.M = q.M;
    o.max_tiles = max_tiles;
    o.R = q.R;
    o.L = q.L;
    o.status = q.status;
    e = bf16_map(&maps.src[0], q.dy, N, q.M, 0, q.lddy, kOuterRows);
    if (e == cudaSuccess) e = bf16_map(&maps.src[1], q.x, K, q.M, 0, q.ldx, kOuterRows);
    if (e == cudaSuccess) e = bf16_map(&maps.rows[0], q.dy, N, q.M, 0, q.lddy, 1);
    if (e == cudaSuccess) e = bf16_map(&maps.rows[1], q.x, K, q.M, 0, q.ldx, 1);
    if (e == cudaSuccess) e = bf16_map(&maps.v[0], vt, q.R, rows, TERMS, q.R, kOuterRows);
    if (e == cudaSuccess) e = bf16_map(&maps.v[1], vdt, q.R, rows, TERMS, q.R, kOuterRows);
    if (e == cudaSuccess)
      e = by_rank(q.R, [&](auto rt) {
        return run_outer<decltype(rt)::value, TERMS>(maps, o, stream);
      });
  }
  if (e == cudaSuccess && q.dx != nullptr) {
    const ExpandArgs x = {nullptr, vdt, q.A, nullptr, q.plan, q.base, q.ld_base, q.dx, q.lddx,
                          q.M, K, q.R, q.L, q.status};
    e = by_rank_fine(q.R, [&](auto rt) {
      return run_expand<decltype(rt)::value, true, false>(x, stream);
    });
  }
  return e;
}

}  // namespace

size_t lora_plan_words(int64_t M, int32_t L) {
  return static_cast<size_t>(plan_recs_at(L) + kRecWords * plan_max_tiles(M, L));
}

size_t lora_workspace_bytes(int64_t M, int32_t R, int32_t L, bool f32) {
  return static_cast<size_t>(plan_max_tiles(M, L)) * kTileRows * R * 2 * 2 * (f32 ? 3 : 1);
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
  const ContractArgs c = {nullptr, q.plan, q.t, nullptr, nullptr, nullptr,
                          q.M, plan_max_tiles(q.M, q.L), static_cast<int32_t>(q.K), q.R, q.L,
                          q.status};
  const ExpandArgs e = {q.t, nullptr, q.B, q.scale, q.plan, q.base, q.ld_base, q.y, q.ldy, q.M,
                        static_cast<int32_t>(q.N), q.R, q.L, q.status};
  const cudaError_t err = by_rank(q.R, [&](auto rt) {
    return run_contract<decltype(rt)::value, false, 0>(q.x, q.ldx, q.A, c, stream);
  });
  if (err != cudaSuccess) return err;
  return by_rank_fine(q.R, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    return q.f32 ? run_expand<RT, false, true>(e, stream) : run_expand<RT, false, false>(e, stream);
  });
}

cudaError_t launch_lora_backward(const LoraRequest &q, cudaStream_t stream) {
  return q.f32 ? run_backward<3>(q, stream) : run_backward<1>(q, stream);
}

}  // namespace sq
