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
// Byte offset of 16-byte chunk c (0..7) of row r in a tile of 128-byte rows with
// 128-byte swizzling, as TMA writes it and tcgen05 reads it.
__device__ __forceinline__ uint32_t swz128(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// Scattered rows come by plain asynchronous copies of a whole warp; their
// arrival is announced two stages late, when the next two stages' copies are
// already under way.  (TMA can gather four rows by number, but 110 MB of rows
// took 72 us that way, against 43 us in boxes.)
struct LateArrival {
  uint64_t *older = nullptr, *newer = nullptr;  // stages whose copies are under way
  template <int KEEP>
  __device__ __forceinline__ void arrive(int lane, uint64_t *bar) {
    if (bar == nullptr) return;
    cp_async_wait<KEEP>();
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  // this stage's copies were just committed
  __device__ __forceinline__ void push(int lane, uint64_t *bar) {
    arrive<2>(lane, older);
    older = newer;
    newer = bar;
  }
  __device__ __forceinline__ void catch_up(int lane) {
    arrive<1>(lane, older);
    arrive<0>(lane, newer);
    older = newer = nullptr;
  }
};

// Sum over blocks lo .. hi (at most 8) of a cluster of the four floats at
// `at`(block) in each one's `part`, in block order, all loads in flight at once.
template <typename At>
__device__ __forceinline__ float4 cluster_sum(cg::cluster_group &cluster, float *part, int lo,
                                              int hi, At &&at) {
  float4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (lo + k <= hi)
      v[k] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(part, lo + k) + at(lo + k));
  }
  float4 s = v[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    s.x += v[k].x;
    s.y += v[k].y;
    s.z += v[k].z;
    s.w += v[k].w;
  }
  return s;
}

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
// dimension: TMA brings the tile's rows as a box, 64 columns a stage, where they
// are neighbours (else a warp copies them), and the weight's box beside them;
// one thread issues tcgen05.mma (M = 128, N = RT, sums in tensor memory), so that
// reading the rows costs the SM next to no instructions.  The blocks of a cluster hold the slices of one tile and add
// their partial sums through distributed shared memory in a fixed order.  The
// forward pass stores t by row in fp32; the backward pass stores dt, and beside
// it t, as bf16 terms by tile, 128 rows each with zeros past the tile's last:
// the operand that the outer products and dx read.
struct ContractArgs {
  const uint16_t *in;  // as tm_in
  int64_t ld;
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
    prefetch_tmap(&tm_in);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, RT);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_dependency_launch();

  // A fitting plan has a record for every block of the grid; the blocks of a
  // cluster share their tile and so their way through this kernel.
  int4 tile = make_int4(p.L, 0, 0, 0);
  const int32_t *rec = p.plan + plan_recs_at(p.L) + static_cast<int64_t>(blockIdx.x) * kRecWords;
  if (plan_fits(p.plan, p.M, p.L, p.status) && static_cast<int>(blockIdx.x) < p.plan[3])
    tile = *reinterpret_cast<const int4 *>(rec);
  const int bin = tile.x, count = tile.y;
  const bool run = tile.w != 0;  // neighbouring rows
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], run ? 1 : 2);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (bin < p.L) {
    const int slice = ((p.C + slices - 1) / slices + 63) / 64 * 64;
    const int c_lo = rank * slice;
    const int c_hi = c_lo + slice < p.C ? c_lo + slice : p.C;
    const int steps = c_hi > c_lo ? (c_hi - c_lo + 63) / 64 : 0;
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      // Rows past the tile's last are the next ones of a box, or left out:
      // what stands there only meets sums that are not stored.
      const int first = rec[4];
      int32_t rows[kTileRows / 4];  // scattered: this lane copies rows 4 i + lane / 8
#pragma unroll
      for (int i = 0; i < kTileRows / 4; ++i) rows[i] = run ? 0 : rec[4 + i * 4 + (lane >> 3)];
      const uint32_t bytes = (run ? S::kIn : 0) + S::kW;
      uint32_t armed = 0, armed_parity = 0;
      LateArrival late;
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
            if (run) tma_load_2d(in, &tm_in, &full[st], c0, first);
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
        if (!run) {
          const int c = lane & 7, col = c0 + c * 8;
          const bool in_cols = col < p.C;
          const uint32_t to = smem_u32(in);
#pragma unroll
          for (int i = 0; i < kTileRows / 4; ++i) {
            if (i * 4 >= count) break;
            const int r = i * 4 + (lane >> 3);
            if (r < count)
              cp_async16(to + swz128(r, c), p.in + rows[i] * p.ld + (in_cols ? col : 0), in_cols);
          }
          cp_async_commit();
          late.push(lane, &full[st]);
        }
      }
      late.catch_up(lane);
      // never leave with a copy in flight into this block's shared memory
      cp_async_wait<0>();
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
        s = slices > 1 ? cluster_sum(cluster, part, 0, slices - 1, [&](int) { return r * PS + j; })
                       : *reinterpret_cast<const float4 *>(part + r * PS + j);
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
// neighbours.  The products add onto base in the accumulators (the scale is in
// t), so that an element costs its two conversions and no arithmetic.  Column 32 b + 8 c + 2 j + e is
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
  const int my_col = wn * (SLAB / 2) + c8;
  int l_tile = tile0, l_slab = slab0;
  const uint8_t *l_base[2] = {nullptr, nullptr};  // nullptr: zeros
  const uint16_t *l_w = nullptr;                  // nullptr: no adapter
  auto next_tile = [&]() {
    const int32_t *rec = recs + static_cast<int64_t>(l_tile) * kRecWords;
    const int bin = rec[0], count = rec[1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = wm * 16 + g + h * 8;
      l_base[h] = p.base != nullptr && r < count
                      ? static_cast<const uint8_t *>(p.base) +
                            (rec[4 + r] * p.ld_base + l_slab * SLAB + my_col) * E
                      : nullptr;
    }
    l_w = bin < p.L ? p.w + static_cast<int64_t>(bin) * p.R * p.C : nullptr;
  };
  auto load = [&](int stage) {
    const uint32_t sw = sm + S::kT + stage * S::kStage;
    const uint32_t sb = sw + S::kW + tid * 16;
    const int left = p.C - l_slab * SLAB;  // columns from this slab on
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const bool ok = l_base[h] != nullptr && my_col + b * 32 < left;
        const uint8_t *src = ok ? l_base[h] + b * 32 * E : reinterpret_cast<const uint8_t *>(p.w);
#pragma unroll
        for (int q = 0; q < Q; ++q)
          cp_async16(sb + ((h * NB + b) * Q + q) * kExpandThreads * 16, ok ? src + q * 16 : src, ok);
      }
      if (l_base[h] != nullptr) l_base[h] += SLAB * E;
    }
    if (l_w != nullptr) {
      if constexpr (!TRANS) {
        constexpr int PER = RT / 8;
        const uint16_t *w = l_w + static_cast<int64_t>(l_slab) * SLAB * p.R;
#pragma unroll
        for (int k = tid; k < SLAB * PER; k += kExpandThreads) {
          const int r = k / PER, cc = k % PER;
          const int at = (r & ~31) | (((r >> 1) & 3) << 3) | (((r >> 3) & 3) << 1) | (r & 1);
          const bool ok = r < left && cc * 8 < p.R;
          cp_async16(sw + at * S::kWRow + cc * 16, ok ? w + r * p.R + cc * 8 : p.w, ok);
        }
      } else {
        constexpr int PER = SLAB / 2;  // pairs of columns
        const uint16_t *w = l_w + l_slab * SLAB;
#pragma unroll 8
        for (int k = tid; k < RT * PER; k += kExpandThreads) {
          const int r = k / PER, cc = k % PER;
          const int at = (cc & ~15) | ((cc & 3) << 2) | ((cc >> 2) & 3);
          const bool ok = r < p.R && cc * 2 < left;
          cp_async4(sw + r * S::kWRow + at * 4,
                    ok ? w + static_cast<int64_t>(r) * p.C + cc * 2 : p.w, ok);
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
  uint8_t *dst[2] = {nullptr, nullptr};  // nullptr: no row
  bool fresh = true;
  for (int i = 0; i < mine; ++i) {
    if (fresh) {
      const int32_t *rec = recs + static_cast<int64_t>(tile) * kRecWords;
      bin = rec[0];
      count = rec[1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = wm * 16 + g + h * 8, row = rec[4 + r];
        dst[h] = r < count && store_ok(p.status, row >= 0 && row < p.M)
                     ? static_cast<uint8_t *>(p.out) + (row * p.ld_out + slab * SLAB + my_col) * E
                     : nullptr;
      }
      if (i > 0) __syncthreads();  // the last tile's t is no longer read
      if (bin < p.L) {
        const float f = p.scale ? p.scale[bin] : 1.0f;
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
            v = make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
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
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const uint4 v = *reinterpret_cast<const uint4 *>(
                st + S::kW + (((h * NB + b) * Q + q) * kExpandThreads + tid) * 16);
            const uint32_t o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (F32) {
                acc[b * 4 + q * 2 + j / 2][2 * h + j % 2] = __uint_as_float(o[j]);
              } else {
                acc[b * 4 + j][2 * h] = bf16_lo(o[j]);
                acc[b * 4 + j][2 * h + 1] = bf16_hi(o[j]);
              }
            }
          }
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
      const int left = p.C - slab * SLAB;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (dst[h] == nullptr || my_col + b * 32 >= left) continue;
          uint32_t o[4 * Q];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = acc[b * 4 + j][2 * h], y = acc[b * 4 + j][2 * h + 1];
            if constexpr (F32) {
              o[2 * j] = __float_as_uint(x);
              o[2 * j + 1] = __float_as_uint(y);
            } else {
              o[j] = bf16x2(x, y);
            }
          }
          uint4 *to = reinterpret_cast<uint4 *>(dst[h] + b * 32 * E);
#pragma unroll
          for (int q = 0; q < Q; ++q)
            to[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (dst[h] != nullptr) dst[h] += SLAB * E;
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
// scale) and dA[a][j][k] (src x, v dt, f = 1, stored transposed).  A cluster
// takes a slab of 128 columns c; its blocks take equal shares of the row tiles
// of all adapters in order, 64 rows a stage: src's rows as a TMA box where 64
// neighbours are the adapter's (else a warp copies them) and v's box; both are
// operands whose rows run along the contraction, M = 128 columns of src by N =
// RT, sums in tensor memory, one buffer in use and one being stored.  v is zero
// in the rows past a tile's last, where src repeats a row of the tile.
// An adapter whose tiles lie in one block goes straight to memory.  A block
// shares at most its first and its last adapter with its neighbours: those
// partial sums meet in distributed shared memory, added in block order.
struct OuterSide {
  const uint16_t *src;  // as the side's map
  int64_t ld;
  const float *scale;   // nullptr: 1
  void *out;
  int32_t C;
  int32_t transposed;   // out [R][C] instead of [C][R]
};
struct OuterArgs {
  OuterSide side[2];
  int32_t slabs0;  // slabs of side 0
  const int32_t *plan;
  int64_t M;
  int32_t R, L;
  int *status;
};
struct OuterMaps {
  CUtensorMap src[2], v[2];
};

constexpr int kOuterThreads = 192;  // producer, MMA issuer, four storing warps
constexpr int kOuterSlab = 128;
constexpr int kOuterRows = 64;  // a stage

template <int RT, int TERMS>
struct OuterSmem {
  static constexpr int kSrc = kOuterRows * kOuterSlab * 2;  // two boxes of 64 columns
  static constexpr int kV = TERMS * kOuterRows * RT * 2;
  static constexpr int kStage = kSrc + kV;
  static constexpr int kStages = 4 * kStage <= 104 * 1024 ? 4 : 3;
  static constexpr int kPartRow = RT + 4;  // floats
  static constexpr int kPart = kOuterSlab * kPartRow * 4;
  static constexpr int kData = kStages * kStage > 2 * kPart ? kStages * kStage : 2 * kPart;
  static constexpr int kBars = (kData + 15) / 16 * 16;
  static constexpr int kBytes = kBars + (2 * kStages + 5) * 8 + kStages * 4 + 16 + 1024;
  static_assert(kBytes <= 232448, "dynamic shared memory above the per-block limit");
  // blocks that share an SM
  static constexpr int kPerSm = 2 * (kBytes + 1024) <= 228 * 1024 ? 2 : 1;
  static_assert(kPerSm * 2 * RT <= 512, "tensor memory of an SM");
};

enum { kStageFirst = 1, kStageLast = 2, kStageEnd = 4 };

template <bool F32>
__device__ __forceinline__ void store_grad(void *out, int64_t at, float v) {
  if constexpr (F32)
    static_cast<float *>(out)[at] = v;
  else
    static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
}

template <int RT, int TERMS>
__global__ void __launch_bounds__(kOuterThreads, OuterSmem<RT, TERMS>::kPerSm)
    lora_outer_kernel(const __grid_constant__ OuterMaps maps, const OuterArgs p) {
  using S = OuterSmem<RT, TERMS>;
  constexpr int STAGES = S::kStages;
  constexpr bool F32 = TERMS > 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *empty = full + STAGES;
  uint64_t *acc_full = empty + STAGES;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *done = acc_empty + 2;
  volatile int *meta = reinterpret_cast<volatile int *>(done + 1);  // [STAGES]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1) + STAGES;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int shares = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slab = static_cast<int>(blockIdx.x) / shares;
  const bool second = slab >= p.slabs0;
  const OuterSide sd = second ? p.side[1] : p.side[0];
  const CUtensorMap *tm_src = second ? &maps.src[1] : &maps.src[0];
  const CUtensorMap *tm_v = second ? &maps.v[1] : &maps.v[0];
  const int c0 = (slab - (second ? p.slabs0 : 0)) * kOuterSlab;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(tm_src);
    prefetch_tmap(tm_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * RT);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const bool fits = plan_fits(p.plan, p.M, p.L, p.status);
  const int32_t *tile_at = p.plan + 4;
  const int32_t *recs = p.plan + plan_recs_at(p.L);
  const int tiles = fits ? tile_at[p.L] : 0;  // of rows with an adapter
  const int holders = tiles < shares ? tiles : shares;  // blocks with any tile
  auto first_tile = [&](int r) {  // of block r of the cluster
    return r < holders ? static_cast<int>(static_cast<int64_t>(tiles) * r / holders) : tiles;
  };
  const int t_lo = first_tile(rank), t_hi = first_tile(rank + 1);
  auto bin_of = [&](int tile) { return recs[static_cast<int64_t>(tile) * kRecWords]; };
  grid_dependency_wait();

  const int cols = sd.C - c0 < kOuterSlab ? sd.C - c0 : kOuterSlab;
  float keep[RT];  // storing warps: the sums of a first adapter that is shared
  bool kept = false, last_shared = false, ok_all = true;
  uint32_t last_buf = 0;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t armed = 0, armed_parity = 0;
    LateArrival late;
    int step = 0;
    bool ok = true;
    // takes the next stage; lane 0 then announces `bytes` of TMA to come
    auto take = [&](int flags, uint32_t bytes) -> int {
      const int st = step % STAGES;
      const uint32_t phase = (step / STAGES) & 1;
      ++step;
      if (lane == 0) {
        ok = bounded_wait(&empty[st], phase ^ 1, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT);
        if (ok) {
          meta[st] = flags;
          mbar_arrive_expect_tx(&full[st], bytes);
          armed |= 1u << st;
          armed_parity = (armed_parity & ~(1u << st)) | (phase << st);
        }
      }
      ok = __shfl_sync(~0u, ok, 0);
      return st;
    };
    const bool wide = c0 + 64 < sd.C;  // no box past the last column
    // records are read two tiles ahead: {bin, rows, -, neighbours} and the row
    // numbers, 32 k + l in lane l
    struct Record {
      int4 h;
      int32_t rows[4];
    };
    auto read = [&](int tile, Record &r) {
      if (tile >= t_hi) return;
      const int32_t *rec = recs + static_cast<int64_t>(tile) * kRecWords;
      r.h = *reinterpret_cast<const int4 *>(rec);
#pragma unroll
      for (int k = 0; k < 4; ++k) r.rows[k] = rec[4 + 32 * k + lane];
    };
    Record now = {make_int4(-1, 0, 0, 0), {0, 0, 0, 0}}, next = now, after = now;
    int bin_before = -1;
    read(t_lo, now);
    read(t_lo + 1, next);
    for (int tile = t_lo; tile < t_hi && ok; ++tile) {
      read(tile + 2, after);
      const int4 h = now.h;
      const int first_row = __shfl_sync(~0u, now.rows[0], 0);
      const int halves = (h.y + kOuterRows - 1) / kOuterRows;
      const bool head = h.x != bin_before;
      const bool tail = tile + 1 == t_hi || next.h.x != h.x;
      for (int q = 0; q < halves && ok; ++q) {
        const bool box = h.w != 0 && (q + 1) * kOuterRows <= h.y;
        const int st = take((head && q == 0 ? kStageFirst : 0) |
                                (tail && q == halves - 1 ? kStageLast : 0),
                            S::kV + (box ? (wide ? 2 : 1) * 8192 : 0));
        if (!ok) break;
        uint8_t *src = smem + st * S::kStage;
        if (lane == 0) {
          if (box) {
            const int row = first_row + q * kOuterRows;
            tma_load_2d(src, tm_src, &full[st], c0, row);
            if (wide) tma_load_2d(src + 8192, tm_src, &full[st], c0 + 64, row);
          }
#pragma unroll
          for (int s = 0; s < TERMS; ++s)
#pragma unroll
            for (int b = 0; b < RT / 64; ++b)
              tma_load_3d(src + S::kSrc + (s * (RT / 64) + b) * 8192, tm_v, &full[st], b * 64,
                          tile * kTileRows + q * kOuterRows, s);
        }
        if (box) {
          late.catch_up(lane);
          if (lane == 0) mbar_arrive(&full[st]);
        } else {
          const int c = lane & 15, col = c0 + c * 8;
          const uint32_t to = smem_u32(src) + (c >> 3) * 8192;
          const bool in_cols = col < sd.C;
          int32_t rows[kOuterRows / 2];  // all exchanged before the first copy
#pragma unroll
          for (int i = 0; i < kOuterRows / 2; ++i)
            rows[i] = __shfl_sync(~0u, q == 0 ? now.rows[i / 16] : now.rows[2 + i / 16],
                                  (i * 2 + (lane >> 4)) & 31);
          if (c < 8 || wide) {
#pragma unroll
            for (int i = 0; i < kOuterRows / 2; ++i)
              cp_async16(to + swz128(i * 2 + (lane >> 4), c & 7),
                         sd.src + rows[i] * sd.ld + (in_cols ? col : 0), in_cols);
          }
          cp_async_commit();
          late.push(lane, &full[st]);
        }
      }
      bin_before = h.x;
      now = next;
      next = after;
    }
    late.catch_up(lane);
    if (ok) {
      const int st = take(kStageEnd, 0);
      if (ok && lane == 0) mbar_arrive(&full[st]);
    }
    // never leave with a copy in flight into this block's shared memory
    cp_async_wait<0>();
    if (lane == 0)
      for (int s = 0; s < STAGES; ++s)
        if (armed & (1u << s)) mbar_wait(&full[s], (armed_parity >> s) & 1u, kBoundedWaitNs);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(kOuterSlab, RT) | kIdescTransA | kIdescTransB;
      uint32_t seg = 0;
      for (int step = 0;; ++step) {
        const int st = step % STAGES;
        if (!bounded_wait(&full[st], (step / STAGES) & 1, abort_flag, p.status,
                          SQ_ERR_DEVICE_TIMEOUT))
          break;
        const int flags = meta[st];
        if (flags & kStageEnd) break;
        const uint32_t acc = tmem + (seg & 1) * RT;
        if (flags & kStageFirst)
          if (!bounded_wait(&acc_empty[seg & 1], ((seg >> 1) & 1) ^ 1, abort_flag, p.status,
                            SQ_ERR_DEVICE_TIMEOUT))
            break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + st * S::kStage), sb = sa + S::kSrc;
#pragma unroll
        for (int q = TERMS - 1; q >= 0; --q)
#pragma unroll
          for (int kk = 0; kk < kOuterRows / 16; ++kk)
            mma_bf16_tc(acc, sdesc_mnmajor_sw128(sa + kk * 2048, 8192),
                        sdesc_mnmajor_sw128(sb + q * (RT / 64) * 8192 + kk * 2048, 8192), idesc,
                        !(flags & kStageFirst) || kk > 0 || q < TERMS - 1);
        mma_commit(&empty[st]);
        if (flags & kStageLast) {
          mma_commit(&acc_full[seg & 1]);
          ++seg;
        }
      }
      mma_commit(done);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ storing warps
    // thread: column c of the slab, sums over all j
    const int c = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t seg = 0;
    for (int tile = t_lo; tile < t_hi; ++seg) {
      const int bin = bin_of(tile);
      const int lo = tile_at[bin], hi = tile_at[bin + 1];
      const bool whole = lo >= t_lo && hi <= t_hi;
      const bool first = tile == t_lo;
      tile = hi < t_hi ? hi : t_hi;
      ok_all = bounded_wait(&acc_full[seg & 1], (seg >> 1) & 1, abort_flag, p.status,
                            SQ_ERR_DEVICE_TIMEOUT);
      if (!ok_all) break;
      tc_fence_after();
      const uint32_t acc = tmem + (seg & 1) * RT + lanes;
      if (!whole && !first) {  // the last one, shared: stays where it is
        last_shared = true;
        last_buf = seg & 1;
        break;
      }
      if (whole) {
        const float f = sd.scale ? sd.scale[bin] : 1.0f;
        const int64_t obase = static_cast<int64_t>(bin) * p.R * sd.C;
#pragma unroll
        for (int j0 = 0; j0 < RT; j0 += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_32x32b_x32(acc + j0, r);
          tmem_ld_wait();
          if (c < cols && store_ok(p.status, c0 + c < sd.C)) {
            if (sd.transposed) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j0 + j < p.R)
                  store_grad<F32>(sd.out, obase + static_cast<int64_t>(j0 + j) * sd.C + c0 + c,
                                  f * __uint_as_float(r[j]));
            } else {
              const int64_t at = obase + static_cast<int64_t>(c0 + c) * p.R + j0;
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                if (j0 + j < p.R) {  // R % 8 == 0
                  float v[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) v[e] = f * __uint_as_float(r[j + e]);
                  if constexpr (F32) {
                    float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(sd.out) + at + j);
                    to[0] = make_float4(v[0], v[1], v[2], v[3]);
                    to[1] = make_float4(v[4], v[5], v[6], v[7]);
                  } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(sd.out) + at + j) =
                        make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                                   bf16x2(v[6], v[7]));
                  }
                }
            }
          }
        }
      } else {
#pragma unroll
        for (int j0 = 0; j0 < RT; j0 += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_32x32b_x32(acc + j0, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) keep[j0 + j] = __uint_as_float(r[j]);
        }
        kept = true;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[seg & 1]);
    }
  }
  const bool ok = bounded_wait(done, 0, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT) && ok_all;
  tc_fence_after();
  __syncthreads();  // nothing reads or fills the stages any more

  // partial sums of the first (0) and the last (1) adapter, [128][RT + 4]
  constexpr int PS = S::kPartRow;
  float *part = reinterpret_cast<float *>(smem);
  if (warp >= 2) {
    const int c = (warp & 3) * 32 + lane;
    if (kept) {
#pragma unroll
      for (int j = 0; j < RT; j += 4)
        *reinterpret_cast<float4 *>(part + c * PS + j) =
            make_float4(keep[j], keep[j + 1], keep[j + 2], keep[j + 3]);
    }
    if (last_shared) {
      float *to = part + kOuterSlab * PS + c * PS;
#pragma unroll
      for (int j0 = 0; j0 < RT; j0 += 32) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(tmem + last_buf * RT + (static_cast<uint32_t>((warp & 3) * 32) << 16) + j0,
                           r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<uint4 *>(to + j0 + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
      }
    }
  }
  if (shares > 1) {
    cluster.sync();
    if (t_lo < t_hi && ok) {
      const int b_first = bin_of(t_lo), b_last = bin_of(t_hi - 1);
      for (int k = 0; k < 2; ++k) {
        const int bin = k == 0 ? b_first : b_last;
        if (k == 1 && b_last == b_first) break;
        const int lo = tile_at[bin], hi = tile_at[bin + 1];
        if (lo >= t_lo && hi <= t_hi) continue;  // all here: stored
        // the blocks that hold tiles of this adapter
        int r_lo = rank, r_hi = rank;
        while (r_lo > 0 && first_tile(r_lo) > lo) --r_lo;
        while (r_hi + 1 < holders && first_tile(r_hi + 1) < hi) ++r_hi;
        const float f = sd.scale ? sd.scale[bin] : 1.0f;
        const int64_t obase = static_cast<int64_t>(bin) * p.R * sd.C;
        const int quads = p.R / 4, n_out = cols * quads, n_blocks = r_hi - r_lo + 1;
        for (int e = (rank - r_lo) * kOuterThreads + threadIdx.x; e < n_out;
             e += n_blocks * kOuterThreads) {
          const int c = sd.transposed ? e % cols : e / quads;
          const int j = (sd.transposed ? e / cols : e % quads) * 4;
          // the adapter is a block's first unless the block begins before it
          const float4 s = cluster_sum(cluster, part, r_lo, r_hi, [&](int r) {
            return (first_tile(r) < lo ? kOuterSlab * PS : 0) + c * PS + j;
          });
          if (!store_ok(p.status, j + 4 <= p.R && c0 + c < sd.C)) continue;
          const float v[4] = {f * s.x, f * s.y, f * s.z, f * s.w};
          if (sd.transposed) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              store_grad<F32>(sd.out, obase + static_cast<int64_t>(j + q) * sd.C + c0 + c, v[q]);
          } else {
            const int64_t at = obase + static_cast<int64_t>(c0 + c) * p.R + j;
            if constexpr (F32)
              *reinterpret_cast<float4 *>(static_cast<float *>(sd.out) + at) =
                  make_float4(v[0], v[1], v[2], v[3]);
            else
              *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(sd.out) + at) =
                  make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
          }
        }
      }
    }
  }
  // adapters without rows: zeros
  if (fits)
    for (int bin = rank; bin < p.L; bin += shares) {
      if (tile_at[bin] != tile_at[bin + 1]) continue;
      const int64_t obase = static_cast<int64_t>(bin) * p.R * sd.C;
      for (int e = threadIdx.x; e < cols * p.R; e += kOuterThreads) {
        const int64_t at = sd.transposed
                               ? obase + static_cast<int64_t>(e / cols) * sd.C + c0 + e % cols
                               : obase + static_cast<int64_t>(c0) * p.R + e;
        if (store_ok(p.status, at < (static_cast<int64_t>(bin) + 1) * p.R * sd.C))
          store_grad<F32>(sd.out, at, 0.0f);
      }
    }
  if (shares > 1) cluster.sync();  // no block leaves while its sums are read

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * RT);
  }
}

// ------------------------------------------------------------------ host side
// Launch with dynamic shared memory and clusters of `cluster` blocks along the
// grid's dimension `dim` (0 x, 1 y, 2 z).  Every kernel here waits for the one
// ahead of it in the stream (programmatic dependent launch) before it reads
// what that one may have written.
//
// By default the driver gives an SM as much shared memory as one block of the
// kernel needs, not as much as would hold two or three: asking for all of it
// doubles (triples) the blocks that run at once.
template <auto Kernel>
cudaError_t allow_smem(int smem) {
  static bool set[64] = {};  // per kernel and device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) set[dev] = true;
  return e;
}

template <auto Kernel, typename... Args>
cudaError_t launch(dim3 grid, int threads, int smem, int cluster, int dim, cudaStream_t stream,
                   const Args &...args) {
  cudaError_t e = allow_smem<Kernel>(smem);
  if (e != cudaSuccess) return e;
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
cudaError_t run_contract(const uint16_t *w, const ContractArgs &a, cudaStream_t stream) {
  CUtensorMap tm_in, tm_w;
  cudaError_t e = bf16_map(&tm_in, a.in, a.C, a.M, 0, a.ld, kTileRows);
  if (e == cudaSuccess)
    e = TRANS ? bf16_map(&tm_w, w, a.R, a.C, a.L, a.R, 64)
              : bf16_map(&tm_w, w, a.C, a.R, a.L, a.C, RT);
  if (e != cudaSuccess) return e;
  // Slices of the contracted dimension: as many as let all tiles run at once
  // (two blocks per SM), none shorter than 256 columns.
  int slices = 1;
  while (slices < 8 && a.C >= 256 * slices * 2 && a.max_tiles * slices * 2 <= 2 * sm_count())
    slices *= 2;
  return launch<lora_contract_kernel<RT, TRANS, TERMS>>(
      dim3(static_cast<unsigned>(a.max_tiles), slices), kContractThreads,
      ContractSmem<RT>::kBytes, slices, 1, stream, tm_in, tm_w, a);
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
  using S = OuterSmem<RT, TERMS>;
  const int slabs = a.slabs0 + (a.side[1].C + kOuterSlab - 1) / kOuterSlab;
  // Blocks of a slab: as many (up to the portable cluster size, and one for each
  // two full row tiles) as let all slabs run at once.  A cluster lies within one
  // of the GPU's partitions, which leaves some places empty: 60 slabs by 4 take
  // 58 us, by 7 (three blocks per SM) two rounds and 80 us.
  int shares = 1;
  for (int n = 2; n <= 8 && a.M >= 2 * kTileRows * n; ++n)
    if (static_cast<int64_t>(slabs) * n * 16 <= static_cast<int64_t>(S::kPerSm) * sm_count() * 15)
      shares = n;
  return launch<lora_outer_kernel<RT, TERMS>>(dim3(slabs * shares), kOuterThreads, S::kBytes,
                                              shares, 0, stream, maps, a);
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
  const ContractArgs c = {q.dy, q.lddy, q.scale, q.plan, nullptr, q.t, vt, vdt,
                          q.M, max_tiles, N, q.R, q.L, q.status};
  cudaError_t e = by_rank(q.R, [&](auto rt) {
    return run_contract<decltype(rt)::value, true, TERMS>(q.B, c, stream);
  });
  if (e == cudaSuccess && q.dA != nullptr) {
    OuterMaps maps;
    OuterArgs o = {};
    o.side[0] = {q.dy, q.lddy, q.scale, q.dB, N, 0};
    o.side[1] = {q.x, q.ldx, nullptr, q.dA, K, 1};
    o.slabs0 = (N + kOuterSlab - 1) / kOuterSlab;
    o.plan = q.plan;
    o.M = q.M;
    o.R = q.R;
    o.L = q.L;
    o.status = q.status;
    e = bf16_map(&maps.src[0], q.dy, N, q.M, 0, q.lddy, kOuterRows);
    if (e == cudaSuccess) e = bf16_map(&maps.src[1], q.x, K, q.M, 0, q.ldx, kOuterRows);
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
  const ContractArgs c = {q.x, q.ldx, nullptr, q.plan, q.t, nullptr, nullptr, nullptr,
                          q.M, plan_max_tiles(q.M, q.L), static_cast<int32_t>(q.K), q.R, q.L,
                          q.status};
  const ExpandArgs e = {q.t, nullptr, q.B, q.scale, q.plan, q.base, q.ld_base, q.y, q.ldy, q.M,
                        static_cast<int32_t>(q.N), q.R, q.L, q.status};
  const cudaError_t err = by_rank(q.R, [&](auto rt) {
    return run_contract<decltype(rt)::value, false, 0>(q.A, c, stream);
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
